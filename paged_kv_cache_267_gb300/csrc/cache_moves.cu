// Moves of cached rows, bit for bit: whole blocks for requests that stop sharing them
// (copy_blocks), and the accepted ones of drafted tokens (compact_cache).
//
// Both are bound by the bytes they move, and where those are few by one launch and two
// dependent round trips (indexes, then rows). A thread moves 16 bytes at a time with
// eight loads in flight.
#include <algorithm>

#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kFlight = 8;  // 16-byte loads in flight a thread
constexpr int kChunk = kThreads * kFlight;  // 16-byte units a CTA moves at once

// CTA (chunk of a block's K or V, pair, layer).
__global__ void __launch_bounds__(kThreads) copy_blocks_kernel(const CopyBlocksArgs a) {
  const int chunk = blockIdx.x % a.chunks;
  const long long rest = blockIdx.x / a.chunks;
  const int pair = static_cast<int>(rest % a.pairs);
  const int plane = static_cast<int>(rest / a.pairs);  // layer, K then V
  griddep_wait();
  const int2 p = a.block_pairs[pair];
  if (p.x < 0 || p.y < 0) return;
  if (p.x >= a.NB || p.y >= a.NB) {
    if (threadIdx.x == 0 && chunk == 0 && plane == 0) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
    return;
  }
  if (p.x == p.y) return;
  const int layer = plane >> 1;
  uint4* const base = reinterpret_cast<uint4*>((plane & 1) ? static_cast<char*>(a.vc) + layer * a.v_layer
                                                           : static_cast<char*>(a.kc) + layer * a.k_layer);
  const uint4* const src = base + static_cast<size_t>(p.x) * a.units;
  uint4* const dst = base + static_cast<size_t>(p.y) * a.units;
  const int at = chunk * kChunk + threadIdx.x;
  uint4 v[kFlight];
#pragma unroll
  for (int i = 0; i < kFlight; ++i)
    if (at + i * kThreads < a.units) v[i] = src[at + i * kThreads];
#pragma unroll
  for (int i = 0; i < kFlight; ++i)
    if (at + i * kThreads < a.units) dst[at + i * kThreads] = v[i];
}

__device__ __forceinline__ int fast_quotient(int x, FastDiv d) {
  return d.mul == 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), d.mul) >> d.shift);
}

// One CTA a (sequence, share of the planes). The rows that move, from where to where, are
// worked out once, into shared memory, and then moved plane by plane, kChunk 16-byte units
// at a time: all of them are loaded before any is stored, and a target lies before every
// later source (the kept tokens ascend), so that passes need no order but their own.
// (A CTA a plane, with 64 of 256 threads at work and the three dependent round trips of
// lengths, list and table in each, took 82 us for 256 sequences of 32 layers.)
__global__ void __launch_bounds__(kThreads) compact_cache_kernel(const CompactArgs a) {
  __shared__ long long s_from[kThreads], s_to[kThreads];  // rows of KV head 0, -1: none
  const int b = blockIdx.x, tid = threadIdx.x;
  griddep_wait();
  const int cap = a.MB * a.bs;
  const int L0 = a.seq_lens[b], L = min(max(L0, 0), cap);
  const int q0 = a.query_start[b], q1 = a.query_start[b + 1];
  const int count = a.num_kept[b];
  const int n = q1 > q0 ? static_cast<int>(min(static_cast<long long>(q1) - q0, 0x7fffffffll)) : 0;
  const int base = L - n;
  const int32_t* kept = a.kept + static_cast<size_t>(b) * a.M;
  const int32_t* table = a.block_tables + static_cast<size_t>(b) * a.MB;
  // the whole list is looked at before anything moves
  bool bad = q1 < q0 || base < 0 || count < 0 || count > min(a.M, n);
  int stay = 0;  // tokens of this thread's that stay in their place
  if (!bad)
    for (int i = tid; i < count; i += kThreads) {
      const int k = kept[i];
      bad = bad || k < 0 || k >= n || (i > 0 && kept[i - 1] >= k);
      stay += k == i;
    }
  bad = __syncthreads_or(bad);
  if (tid == 0 && blockIdx.y == 0) {
    if (L0 != L) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    if (bad) atomicOr(a.err, PA_DEVERR_QUERY);
    const int len = bad ? L : base + count;
    a.lens_out[b] = len;
    if (a.kept_tokens) a.kept_tokens[b] = (len + a.bs - 1) / a.bs * a.bs;
  }
  if (bad) return;
  // (an ascending list stays in place up to its first gap)
  __shared__ int s_stay;
  if (tid == 0) s_stay = 0;
  __syncthreads();
  if (stay) atomicAdd(&s_stay, stay);
  __syncthreads();
  const int units = a.row_units * a.Hkv;
  const long long head = static_cast<long long>(a.bs) * a.row_units;  // units between KV heads
  const int plane0 = blockIdx.y * a.share, planes = min(a.share, 2 * a.layers - plane0);
  for (int i0 = s_stay; i0 < count; i0 += kThreads) {
    const int rows = min(count - i0, kThreads);
    if (tid < rows) {
      auto row_of = [&](int pos) -> long long {
        const int lb = pos / a.bs, blk = table[lb];
        return blk < 0 || blk >= a.NB ? -1 : static_cast<long long>(blk) * a.Hkv * a.bs + (pos - lb * a.bs);
      };
      const long long from = row_of(base + kept[i0 + tid]), to = row_of(base + i0 + tid);
      if (from < 0 || to < 0) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
      s_from[tid] = from;
      s_to[tid] = from < 0 ? -1 : to;
    }
    __syncthreads();
    const int all = planes * rows * units;  // (below 2^31 - kChunk: the launcher sees to it)
    for (int e0 = 0; e0 < all; e0 += kChunk) {
      uint4 v[kFlight];
      uint4* to[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int e = e0 + i * kThreads + tid;
        to[i] = nullptr;
        if (e >= all) continue;
        const int r = fast_quotient(e, a.unit_div), u = e - r * units;
        const int p = static_cast<unsigned>(r) / static_cast<unsigned>(rows), row = r - p * rows;
        const int plane = plane0 + p, layer = plane >> 1;
        const int h = fast_quotient(u, a.row_div), c = u - h * a.row_units;
        if (s_to[row] < 0) continue;
        uint4* const cache = reinterpret_cast<uint4*>(
            (plane & 1) ? static_cast<char*>(a.vc) + layer * a.v_layer : static_cast<char*>(a.kc) + layer * a.k_layer);
        const long long off = h * head + c;
        v[i] = cache[s_from[row] * a.row_units + off];
        to[i] = cache + s_to[row] * a.row_units + off;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (to[i]) *to[i] = v[i];
    }
    __syncthreads();  // the list is written over
  }
}

template <typename K, typename A>
cudaError_t launch(K kernel, dim3 grid, const A& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

int copy_blocks_chunk() { return kChunk; }

cudaError_t copy_blocks_launch(const CopyBlocksArgs& a, cudaStream_t s) {
  const long long grid = static_cast<long long>(a.chunks) * a.pairs * a.layers * 2;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch(copy_blocks_kernel, dim3(static_cast<unsigned>(grid)), a, s);
}

cudaError_t compact_cache_launch(const CompactArgs& a, int num_sms, cudaStream_t s) {
  CompactArgs x = a;
  // as many planes a CTA as leave the GPU a few waves of CTAs
  const int planes = std::max(2 * a.layers, 1);  // (no layers: lengths only)
  const long long ctas = static_cast<long long>(a.B) * planes;
  const long long units = static_cast<long long>(a.row_units) * a.Hkv;
  x.share = static_cast<int>(std::min<long long>(std::max<long long>(ctas / (num_sms * 16ll), 1), planes));
  x.share = static_cast<int>(std::min<long long>(x.share, std::max<long long>(0x7fff0000ll / (kThreads * std::max(units, 1ll)), 1)));
  x.unit_div = fast_div(static_cast<uint32_t>(units));
  x.row_div = fast_div(static_cast<uint32_t>(a.row_units));
  return launch(compact_cache_kernel, dim3(a.B, (planes + x.share - 1) / x.share), x, s);
}

}  // namespace pa
