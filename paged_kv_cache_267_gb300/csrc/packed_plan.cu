// Plan of a ragged step (layout and meaning in packed_plan.cuh): one CTA turns
// query starts and sequence lengths into the items of the attention's CTAs.
// A few thousand integers, bound by its chain of loads, scans and stores.
#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 256;
constexpr unsigned kFull = 0xffffffffu;

// Inclusive scan of x over the block with op (identity `zero`); *total receives the
// whole block's value.
template <typename Op>
__device__ __forceinline__ int scan(int x, int zero, Op op, int* total) {
  __shared__ int s_w[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x = op(x, y);
  }
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  int v = s_w[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v = op(v, y);
  }
  *total = __shfl_sync(kFull, v, 31);
  const int before = __shfl_sync(kFull, v, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // s_w is reused
  return op(x, warp > 0 ? before : zero);
}

__global__ void __launch_bounds__(kThreads, 1) packed_plan_kernel(const PackedPlanArgs a) {
  extern __shared__ int s_dyn[];
  int* s_q = s_dyn;            // [B + 1] query starts, made non-decreasing in [0, T]
  int* s_u = s_dyn + a.B + 1;  // [B + 1] units before each sequence
  __shared__ int s_f[kThreads];  // tiles before each unit of a pass
  __shared__ int s_bin[kBins];
  __shared__ int s_max;
  const int tid = threadIdx.x;
  const int cap = a.MB * a.bs;
  const auto add = [](int x, int y) { return x + y; };
  const auto most = [](int x, int y) { return x > y ? x : y; };
  griddep_launch_dependents();  // the attention sets itself up, then waits
  griddep_wait();               // lengths and starts may be the previous kernel's
  int total;
  for (int b0 = 0, run = 0; b0 <= a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int x = 0;
    if (b <= a.B) {
      const int s = a.query_start[b];
      x = min(max(s, 0), a.T);
      if (s != x) atomicOr(a.err, PA_DEVERR_QUERY);
    }
    const int y = most(scan(x, 0, most, &total), run);
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
      const int n = s_q[b + 1] - s_q[b], L = a.seq_lens[b];
      nu = (n + a.tpu - 1) / a.tpu;
      if (L < 0 || L > cap) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
      if (a.tree && n > 64) atomicOr(a.err, PA_DEVERR_QUERY);
    }
    const int y = scan(nu, 0, add, &total);
    if (b < a.B) s_u[b] = units + y - nu;
    units += total;
  }
  if (tid == 0) s_u[a.B] = units, s_max = 0;
  if (tid < kBins) s_bin[tid] = 0;
  __syncthreads();

  // Unit u as an item with all of its tiles.
  auto unit = [&](int u) -> PackedItem {
    int lo = 0, hi = a.B;  // the last sequence with s_u <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_u[mid] <= u) lo = mid;
      else hi = mid;
    }
    PackedItem it;
    const int b = lo, n = s_q[b + 1] - s_q[b], t0 = (u - s_u[b]) * a.tpu;
    const int L = min(max(a.seq_lens[b], 0), cap);
    it.b = b;
    it.kvh = 0;
    it.row0 = s_q[b] + t0;
    it.ntok = min(a.tpu, n - t0);
    it.first = L - n;
    it.pos0 = it.first + t0;
    // causal: from the first token's window to the last token; tree: from the
    // window of a row with no ancestor to the last drafted token that a bit can name
    it.hi = a.tree ? it.first + min(n, 64) - 1 : it.pos0 + it.ntok - 1;
    const int from = a.tree ? it.first : it.pos0 + 1;
    it.lo = a.window > 0 && from > a.window ? from - a.window : 0;
    it.tile0 = 0;
    it.nt = it.hi >= it.lo ? (it.hi + 1 - (it.lo & ~15) + a.kv - 1) / a.kv : 0;
    it.slot = -1;
    it.pad = 0;
    return it;
  };
  int* const plan = a.plan;
  int2* const ctas = reinterpret_cast<int2*>(plan + packed_ctas_at());
  PackedJoin* const joins = reinterpret_cast<PackedJoin*>(plan + packed_joins_at(a.ctas));
  PackedItem* const items = reinterpret_cast<PackedItem*>(plan + packed_items_at(a.ctas));
  for (int w = tid; w < a.ctas; w += kThreads) {
    ctas[w] = make_int2(0, 0);
    joins[w].n = 0;
  }
  const int out = a.unit_tiles;
  int places = 0;  // of all units of one KV head
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    const int u = u0 + tid;
    const int c = u < units ? out + max(unit(u).nt, 1) : 0;
    scan(c, 0, add, &total);
    places += total;
    if (c > 0) atomicMax(&s_max, c);
  }
  __syncthreads();
  const int longest = s_max;
  const long long all = static_cast<long long>(places) * a.Hkv;
  const int nitems = units * a.Hkv;
  // Whole units, or tiles split evenly? A split takes every CTA the mean, and besides
  // what the partial results and their join cost; whole units take as long as the
  // CTA with the most, which is looked up once they are dealt out.
  const long long mean = (all + a.ctas - 1) / a.ctas;
  const long long split_cost = mean + a.split_tiles;
  bool whole = longest <= split_cost;
  if (whole) {
    // sorted by tiles in kBins steps, most first
    auto bin_of = [&](int nt) {
      return kBins - 1 - static_cast<int>(static_cast<long long>(nt) * (kBins - 1) / longest);
    };
    for (int u = tid; u < units; u += kThreads) atomicAdd(&s_bin[bin_of(unit(u).nt)], 1);
    __syncthreads();
    const int n = tid < kBins ? s_bin[tid] : 0;
    const int y = scan(n, 0, add, &total);
    if (tid < kBins) s_bin[tid] = y - n;
    if (tid == 0) s_max = 0;
    __syncthreads();
    for (int u = tid; u < units; u += kThreads) {
      PackedItem it = unit(u);
      const int at = atomicAdd(&s_bin[bin_of(it.nt)], 1);
      for (int h = 0; h < a.Hkv; ++h) {
        it.kvh = h;
        items[at * a.Hkv + h] = it;
      }
    }
    if (nitems > a.ctas) {
      __syncthreads();
      for (int w = tid; w < a.ctas; w += kThreads) {
        int cost = 0;
        for (int k = 0, i = w; i < nitems; ++k, i = k * a.ctas + ((k & 1) ? a.ctas - 1 - w : w))
          cost += out + max(items[i].nt, 1);
        atomicMax(&s_max, cost);
      }
      __syncthreads();
      whole = s_max <= split_cost;
      __syncthreads();  // before the items are written over
    }
  }
  if (tid == 0) {
    plan[kPkWhole] = whole;
    plan[kPkItems] = nitems;
  }
  if (whole) return;
  const int wsz = static_cast<int>(max(mean, static_cast<long long>(a.min_tiles)));
  int before = 0;  // places of the passes before
  for (int u0 = 0; u0 < units; u0 += kThreads) {
    const int nu = min(units - u0, kThreads);
    const int c = tid < nu ? out + max(unit(u0 + tid).nt, 1) : 0;
    s_f[tid] = before + scan(c, 0, add, &total) - c;
    before += total;
    __syncthreads();
    for (int p = tid; p < nu * a.Hkv; p += kThreads) {
      const int v = p / a.Hkv, h = p - v * a.Hkv;
      PackedItem it = unit(u0 + v);
      it.kvh = h;
      const int nt = it.nt, tiles = max(nt, 1);
      const int f0 = s_f[v] * a.Hkv + h * (out + tiles);  // (below 2^31: the host checks)
      const int g0 = f0 + out, f1 = g0 + tiles;           // its tiles, its end
      const int w0 = g0 / wsz, w1 = (f1 - 1) / wsz;
      const int id = (u0 + v) * a.Hkv + h;
      for (int w = w0; w <= w1; ++w) {
        const int from = max(g0, w * wsz), to = w == w1 ? f1 : (w + 1) * wsz;
        it.tile0 = from - g0;
        it.nt = nt == 0 ? 0 : to - from;
        const bool opens = f0 <= w * wsz;  // the CTA's first: nothing of it lies before
        it.slot = w0 == w1 ? -1 : 2 * w + (opens ? 0 : 1);
        items[id + w] = it;
        if (opens) ctas[w].x = id + w;
        // its last: the next unit's tiles begin behind its end
        if (f1 + out >= (w + 1) * wsz || f1 == all) ctas[w].y = id + w + 1;
      }
      if (w0 != w1) {
        PackedJoin j;
        j.row0 = it.row0;
        j.ntok = it.ntok;
        j.kvh = h;
        j.n = w1 - w0 + 1;
        j.slot0 = 2 * w0 + (f0 <= w0 * wsz ? 0 : 1);
        j.slot1 = 2 * (w0 + 1);
        j.pad[0] = j.pad[1] = 0;
        joins[w0] = j;
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t packed_plan_launch(const PackedPlanArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 2 * (static_cast<size_t>(a.B) + 1) * sizeof(int);  // at most 33 KB
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, packed_plan_kernel, a);
}

}  // namespace pa
