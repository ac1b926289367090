// Plan of a ragged step (layout and meaning in packed_plan.cuh): one CTA turns
// query starts and sequence lengths into the units of the step and each CTA's share.
// A few thousand integers, bound by its chain of loads, block-wide scans and stores, so
// that units are stored once, for all KV heads (an item a pair and 14 dependent loads to
// add up the CTAs' costs had taken 23 us for 256 units).
#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kBins = 256;
constexpr int kSmallUnits = 512;  // fewer units: a small block, whose scans are shorter
constexpr unsigned kFull = 0xffffffffu;

// Inclusive scan of x over the block with op (identity `zero`); *total receives the
// whole block's value.
template <int kThreads, typename T, typename Op>
__device__ __forceinline__ T scan(T x, T zero, Op op, T* total) {
  __shared__ T s_w[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x = op(x, y);
  }
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  T v = lane < kThreads / 32 ? s_w[lane] : zero;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v = op(v, y);
  }
  *total = __shfl_sync(kFull, v, 31);
  const T before = __shfl_sync(kFull, v, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // s_w is reused
  return op(x, warp > 0 ? before : zero);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) packed_plan_kernel(const PackedPlanArgs a) {
  extern __shared__ int s_dyn[];
  int* s_q = s_dyn;             // [B + 1] query starts, made non-decreasing in [0, T]
  int* s_u = s_q + a.B + 1;     // [B + 1] units before each sequence
  int* s_len = s_u + a.B + 1;   // [B] lengths, inside the tables
  __shared__ int s_bin[kBins];
  __shared__ int s_place[kThreads];  // places before the units of a pass
  __shared__ int s_max;
  __shared__ long long s_most;
  const int tid = threadIdx.x;
  const int cap = a.MB * a.bs;
  const auto add = [](auto x, auto y) { return x + y; };
  const auto most = [](int x, int y) { return x > y ? x : y; };
  griddep_launch_dependents();  // the attention sets itself up, then waits
  griddep_wait();               // lengths and starts may be the previous kernel's
  int total;
  for (int b0 = 0, run = 0; b0 <= a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int x = 0;
    if (b <= a.B) {
      const int s = a.query_start[b];
      const int L = b < a.B ? a.seq_lens[b] : 0, M = min(max(L, 0), cap);
      x = min(max(s, 0), a.T);
      if (s != x) atomicOr(a.err, PA_DEVERR_QUERY);
      if (L != M) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
      if (b < a.B) s_len[b] = M;
    }
    const int y = most(scan<kThreads>(x, 0, most, &total), run);
    if (b <= a.B) {
      s_q[b] = y;
      if (y != x) atomicOr(a.err, PA_DEVERR_QUERY);
    }
    run = most(run, total);
  }
  __syncthreads();
  int units = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int nu = 0;
    if (b < a.B) {
      const int n = s_q[b + 1] - s_q[b];
      nu = (n + a.tpu - 1) / a.tpu;
      if (a.tree && n > 64) atomicOr(a.err, PA_DEVERR_QUERY);
    }
    const int y = scan<kThreads>(nu, 0, add, &total);
    if (b < a.B) s_u[b] = units + y - nu;
    units += total;
  }
  if (tid == 0) s_u[a.B] = units, s_max = 0, s_most = 0;
  if (tid < kBins) s_bin[tid] = 0;
  __syncthreads();

  auto unit = [&](int u) -> PackedUnit {
    int lo = 0, hi = a.B;  // the last sequence with s_u <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_u[mid] <= u) lo = mid;
      else hi = mid;
    }
    return packed_unit(lo, u - s_u[lo], s_q[lo], s_q[lo + 1] - s_q[lo], s_len[lo], a.tpu, a.kv, a.window, a.tree);
  };
  auto per_tile = [&](const PackedUnit& it) { return tile_places(it.ntok > a.tpg); };
  auto cost_of = [&](const PackedUnit& it) { return pair_places(it.nt, it.ntok > a.tpg); };
  int* const plan = a.plan;
  int2* const ctas = reinterpret_cast<int2*>(plan + packed_ctas_at());
  PackedJoin* const joins = reinterpret_cast<PackedJoin*>(plan + packed_joins_at(a.ctas));
  auto put = [&](int at, const PackedUnit& it) {
    int4* p = reinterpret_cast<int4*>(plan + packed_units_at(a.ctas)) + 3 * static_cast<size_t>(at);
    p[0] = make_int4(it.b, it.row0, it.ntok, it.pos0);
    p[1] = make_int4(it.first, it.lo, it.hi, it.nt);
    p[2] = make_int4(it.place, 0, 0, 0);
  };

  long long places = 0, sum;  // of all units of one KV head
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    const int u = u0 + tid;
    const int c = u < units ? cost_of(unit(u)) : 0;
    scan<kThreads>(static_cast<long long>(c), 0ll, add, &sum);
    places += sum;
    if (c > 0) atomicMax(&s_max, c);
  }
  __syncthreads();
  const int longest = s_max;
  const long long all = places * a.Hkv;
  const long long pairs = static_cast<long long>(units) * a.Hkv;
  const long long mean = (all + a.ctas - 1) / a.ctas;
  // units by cost, in kBins steps, most first
  auto bin_of = [&](int c) {
    return min(static_cast<int>(static_cast<float>(longest - c) * (static_cast<float>(kBins) / longest)), kBins - 1);
  };
  for (int u = tid; u < units; u += kThreads) atomicAdd(&s_bin[bin_of(cost_of(unit(u)))], 1);
  __syncthreads();
  const int in_bin = tid < kBins ? s_bin[tid] : 0;
  const int upto = scan<kThreads>(in_bin, 0, add, &total);
  // Whole pairs, or places split evenly? A split takes every CTA the mean, and what the
  // partial results and their join cost. Whole pairs, taken most first, take the mean
  // as well, but not less than the longest, nor than k + 1 of the k C-th longest (some
  // CTA has as many of those or longer ones).
  if (tid < kBins && in_bin > 0) {
    const long long r0 = static_cast<long long>(upto - in_bin) * a.Hkv, r1 = static_cast<long long>(upto) * a.Hkv;
    const long long k = (r1 - 1) / a.ctas;
    const int c = longest - static_cast<int>(tid * (static_cast<float>(longest) / kBins));
    if (k * a.ctas >= r0) atomicMax(&s_most, (k + 1) * c);
  }
  if (tid < kBins) s_bin[tid] = upto - in_bin;
  __syncthreads();
  const bool whole = max(mean, s_most) <= mean + a.split_places || all >= 0x7fffffffll - 4096;
  const int wsz = static_cast<int>(max(min(mean, 0x7fffffffll - 4096), static_cast<long long>(a.min_places)));
  if (tid == 0) {
    plan[kPkWhole] = whole;
    plan[kPkPairs] = static_cast<int>(pairs);
    plan[kPkWsz] = wsz;
    plan[kPkNext] = 0;
  }
  for (int w = tid; w < a.ctas; w += kThreads) {
    joins[w].n = 0;
    // (the first CTA's first pair and the last one's end; all others' follow below)
    const bool any = static_cast<long long>(w) * wsz < all, last = static_cast<long long>(w + 1) * wsz >= all;
    if (w == 0 || !any) ctas[w].x = 0;
    if (!any || last) ctas[w].y = any ? static_cast<int>(pairs) : 0;
  }
  if (whole) {
    for (int u = tid; u < units; u += kThreads) {
      const PackedUnit it = unit(u);
      put(atomicAdd(&s_bin[bin_of(cost_of(it))], 1), it);
    }
    return;
  }
  __syncthreads();
  int before = 0;  // places of the passes before, one KV head
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    const int u = u0 + tid, nu = min(units - u0, kThreads);
    PackedUnit it;
    int c = 0;
    if (u < units) {
      it = unit(u);
      c = cost_of(it);
    }
    const int upto_c = scan<kThreads>(c, 0, add, &total);
    s_place[tid] = (before + upto_c - c) * a.Hkv;  // (all places are below 2^31)
    if (u < units) {
      it.place = s_place[tid];
      put(u, it);
    }
    __syncthreads();
    // the CTAs' ends inside this pass's units
    const int from = before * a.Hkv, to = (before + total) * a.Hkv;
    for (int w = tid; w < a.ctas; w += kThreads) {
      const long long at = static_cast<long long>(w) * wsz;
      if (w == 0 || at < from || at >= to) continue;
      int lo = 0, hi = nu;  // the last unit with s_place <= at
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_place[mid] <= at) lo = mid;
        else hi = mid;
      }
      const PackedUnit e = unit(u0 + lo);
      const int per = per_tile(e), nt = max(e.nt, 1), cost = kOutPlaces + nt * per;
      const int x = static_cast<int>(at) - s_place[lo], h = x / cost;
      const int t = tiles_before(x - h * cost - kOutPlaces, nt, per);  // of pair h before the end
      const int p = (u0 + lo) * a.Hkv + h;
      ctas[w].x = t < nt ? p : p + 1;
      ctas[w - 1].y = t > 0 ? p + 1 : p;
      const int g0 = s_place[lo] + h * cost + kOutPlaces;
      if (t > 0 && t < nt && g0 / wsz == w - 1) {  // the pair begins in the CTA before
        PackedJoin j = {};
        j.row0 = e.row0;
        j.ntok = e.ntok;
        j.kvh = h;
        j.n = (g0 + (nt - 1) * per) / wsz - (w - 1) + 1;
        joins[w - 1] = j;
      }
    }
    __syncthreads();
    before += total;
  }
}

}  // namespace

cudaError_t packed_plan_launch(const PackedPlanArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  const bool small = a.T / a.tpu + (a.B < a.T ? a.B : a.T) <= kSmallUnits;
  const auto kernel = small ? packed_plan_kernel<256> : packed_plan_kernel<1024>;
  cfg.blockDim = dim3(small ? 256 : 1024);
  cfg.dynamicSmemBytes = (3 * static_cast<size_t>(a.B) + 2) * sizeof(int);
  if (cfg.dynamicSmemBytes > 32 * 1024) {  // (48 KB, the static part counted)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace pa
