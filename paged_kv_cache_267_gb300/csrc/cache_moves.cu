// Moves of cached rows, bit for bit: whole blocks for requests that stop sharing them
// (copy_blocks), and the accepted ones of drafted tokens (compact_cache).
//
// Both are bound by the bytes they move, and where those are few by one launch and two
// dependent round trips (indexes, then rows). A thread moves 16 bytes at a time with
// eight loads in flight.
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

// One CTA a (sequence, plane): every thread has its 16-byte units of a row of all heads,
// and moves them from kept token to kept token: a target lies before every later source
// (the kept tokens ascend), so a thread's own order is all that is needed.
__global__ void __launch_bounds__(kThreads) compact_cache_kernel(const CompactArgs a) {
  const int b = blockIdx.x, plane = blockIdx.y;
  griddep_wait();
  const int cap = a.MB * a.bs;
  const int L0 = a.seq_lens[b], L = min(max(L0, 0), cap);
  const int q0 = a.query_start[b], q1 = a.query_start[b + 1];
  const int n = max(q1 - q0, 0), base = L - n, count = a.num_kept[b];
  const int32_t* kept = a.kept + static_cast<size_t>(b) * a.M;
  // the whole list is looked at before anything moves
  bool bad = q1 < q0 || base < 0 || count < 0 || count > min(a.M, n);
  if (!bad)
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const int k = kept[i];
      bad = bad || k < 0 || k >= n || (i > 0 && kept[i - 1] >= k);
    }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0 && plane == 0) {
    if (L0 != L) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    if (bad) atomicOr(a.err, PA_DEVERR_QUERY);
    const int len = bad ? L : base + count;
    a.lens_out[b] = len;
    if (a.kept_tokens) a.kept_tokens[b] = (len + a.bs - 1) / a.bs * a.bs;
  }
  if (bad) return;
  const int32_t* table = a.block_tables + static_cast<size_t>(b) * a.MB;
  const int layer = plane >> 1;
  char* const cache = (plane & 1) ? static_cast<char*>(a.vc) + layer * a.v_layer
                                  : static_cast<char*>(a.kc) + layer * a.k_layer;
  const size_t row_bytes = static_cast<size_t>(a.row_units) * 16;
  bool wrong = false;
  // the row of KV head 0 at a position; blocks outside of the pool move nothing
  auto row_of = [&](int pos) -> char* {
    const int lb = pos / a.bs, blk = table[lb];
    if (blk < 0 || blk >= a.NB) {
      wrong = true;
      return nullptr;
    }
    return cache + (static_cast<size_t>(blk) * a.Hkv * a.bs + (pos - lb * a.bs)) * row_bytes;
  };
  const int units = a.row_units * a.Hkv;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    const int h = u / a.row_units, c = u - h * a.row_units;
    const size_t off = static_cast<size_t>(h) * a.bs * row_bytes + static_cast<size_t>(c) * 16;
    for (int i0 = 0; i0 < count; i0 += kFlight) {
      uint4 v[kFlight];
      char* to[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        to[i] = nullptr;
        if (i0 + i >= count) continue;
        const int k = kept[i0 + i];
        if (k == i0 + i) continue;  // in its place already
        const char* from = row_of(base + k);
        to[i] = row_of(base + i0 + i);
        if (!from) to[i] = nullptr;
        if (to[i]) v[i] = *reinterpret_cast<const uint4*>(from + off);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (to[i]) *reinterpret_cast<uint4*>(to[i] + off) = v[i];
    }
  }
  if (wrong) atomicOr(a.err, PA_DEVERR_BLOCK_ID);
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

cudaError_t compact_cache_launch(const CompactArgs& a, cudaStream_t s) {
  return launch(compact_cache_kernel, dim3(a.B, 2 * a.layers), a, s);
}

}  // namespace pa
