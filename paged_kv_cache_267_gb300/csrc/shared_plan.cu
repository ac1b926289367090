// Plan of a shared-prefix decode step (layout and meaning in shared_plan.cuh):
// one CTA turns group starts, prefix lengths and sequence lengths into the
// units, segments and partial slots of the step. A few thousand integers,
// bound by its chain of block-wide scans and its one pass through its
// instructions: 4.7 us from its start to its end for 64 to 256 sequences. It reads
// none of what the write path writes, so it runs while that drains.
#include "pa_internal.h"
#include "ptx.cuh"
#include "shared_plan.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kMostGroups = 4096;  // as the host checks
constexpr unsigned kFull = 0xffffffffu;

// Inclusive scan of x over the block with op (identity `zero`); *total
// receives the whole block's value. ONE: only the first warp has values, and
// only it calls.
template <bool ONE, typename Op>
__device__ __forceinline__ int scan(int x, int zero, Op op, int* total) {
  __shared__ int s_w[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x = op(x, y);
  }
  if constexpr (ONE) {
    *total = __shfl_sync(kFull, x, 31);
    return x;
  }
  if (lane == 31) s_w[warp] = x;
  __syncthreads();
  int v = lane < static_cast<int>(blockDim.x >> 5) ? s_w[lane] : zero;
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

// A group's units, worked out once (every division of a chain of them costs
// about 200 cycles here).
struct Units {
  int nt, nut, up;
  uint32_t up_mul;  // i / up = umulhi(i, up_mul) for i <= 4096; 0: up is 1
};

// How many CTAs (SMs) the prefix kernel's tiles go to. The decode kernel needs
// none of its results and takes the SMs it leaves free, so the step lasts as
// long as the longer of the two,
//   max(a + Tp / n, b + Td / (N - n)),
// with the tiles' times on one SM (measured with both kernels running) and what
// a CTA of each costs once. They are equal where, with c = a - b and
// S = Tp + Td - c N,  c n^2 + S n - Tp N = 0, which is solved without a difference
// of large numbers. Near all SMs, the kernels run better one after the other: with
// 95% of the SMs for a 65536-token document its step took 93 us, with all of them
// first 71. (Every n tried, 32 at once: 1,000 cycles, a tenth of the plan.)
__device__ __forceinline__ int share_sms(const SharedPlanArgs& a, int tiles, int dual, int units, int tails) {
  const float tp = a.cost.dual_ns * dual + a.cost.single_ns * (tiles - dual) + a.cost.unit_ns * units;
  const float td = a.cost.tail_ns * tails, N = a.ctas, c = a.cost.prefix_ns - a.cost.decode_ns;
  const float s = tp + td - c * N, root = sqrtf(fmaxf(s * s + 4.f * c * tp * N, 0.f));
  const int n = static_cast<int>(__fdividef(2.f * tp * N, fmaxf(s + root, 1.f)) + 0.5f);
  return n > a.whole ? a.ctas : max(n, 1);
}

// ONE: up to 31 groups, whose scans are the first warp's alone (a much shorter
// program: most of the time goes by in its one pass through the instructions).
template <bool ONE>
__global__ void __launch_bounds__(kMaxThreads) shared_plan_kernel(const SharedPlanArgs a) {
  extern __shared__ int s_dyn[];
  Units* s_units = reinterpret_cast<Units*>(s_dyn);                // [NG]
  int* s_r0 = s_dyn + 4 * a.NG;  // [NG + 1] group starts, made non-decreasing in [0, B]
  int* s_pre = s_r0 + a.NG + 1;  // [NG] prefix lengths, whole blocks
  int* s_in = s_pre + a.NG;      // [NG] rows that take part, then first flat tile
  int* s_first = s_in + a.NG;    // [NG] the first of them
  int* s_last = s_first + a.NG;  // [NG] and the last
  int* s_base = s_last + a.NG;   // [NG] first slot
  int* s_w0 = s_base + a.NG;     // [NG] first CTA that meets the group
  int* s_lo = s_w0 + a.NG;       // [NG] first position that all taking part attend to
  __shared__ int s_wsz, s_tiles, s_tails, s_dual, s_nunits;
  const int tid = threadIdx.x, nthreads = blockDim.x;
  const int cap = a.MB * a.bs;
  const auto add = [](int x, int y) { return x + y; };
  const auto most = [](int x, int y) { return x > y ? x : y; };
  const bool mine = !ONE || tid < 32;
  const int step = ONE ? 32 : nthreads;
  griddep_launch_dependents();  // the prefix kernel sets itself up, then waits
  // The inputs are not the write path's: planning overlaps it. The workspace
  // it fills was last read by a kernel that an early-launching predecessor
  // has already waited for.
  int len[4];  // this thread's first rows, in flight while the groups are set up
#pragma unroll
  for (int j = 0; j < 4; ++j) len[j] = tid + j * nthreads < a.B ? a.seq_lens[tid + j * nthreads] : 0;
  auto length = [&](int b, int j, bool report = false) -> int {
    const int L = j < 4 ? len[j] : a.seq_lens[b], x = min(max(L, 0), cap);
    if (report && x != L) atomicOr(a.err, PA_DEVERR_SEQ_LEN);
    return x;
  };
  if (tid == 0) s_tails = s_dual = s_nunits = 0;
  int total;
  if (mine) {
    int run = 0;
    for (int g0 = 0; g0 <= a.NG; g0 += step) {
      const int g = g0 + tid;
      int x = 0;
      bool bad = false;
      if (g <= a.NG) {
        const int s = a.group_starts[g];
        const int p = g < a.NG ? a.prefix_lens[g] : 0;
        x = min(max(s, 0), a.B);
        bad = s != x;
        if (g < a.NG) {
          const int q = min(max(p, 0), cap);
          bad = bad || p != q;
          s_pre[g] = q / a.bs * a.bs;
          s_in[g] = 0;
          s_first[g] = a.B;
          s_last[g] = -1;
          s_lo[g] = 0;
        }
      }
      const int y = most(scan<ONE>(x, 0, most, &total), run);
      if (g <= a.NG) {
        s_r0[g] = y;
        bad = bad || y != x;
      }
      if (bad) atomicOr(a.err, PA_DEVERR_GROUP);
      run = most(run, total);
    }
  }
  __syncthreads();
  auto group_of = [&](int b) -> int {  // the group of row b, -1 for none
    if (b < s_r0[0] || b >= s_r0[a.NG]) return -1;
    int lo = 0, hi = a.NG;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_r0[mid] <= b) lo = mid; else hi = mid;
    }
    return lo;
  };
  auto takes_part = [&](int L, int g) -> bool {
    return g >= 0 && s_pre[g] > 0 && L >= s_pre[g] &&
           (a.window == 0 || L <= a.window || L - s_pre[g] <= a.window / 2);
  };
  auto start_of = [&](int L) -> int { return a.window > 0 ? max(L - a.window, 0) : 0; };
  // Rows that take part, by group: a warp's rows are mostly of one group, and
  // are then counted by one lane.
  int tails = 0;  // 16-token tiles of all ranges, of one KV head
  for (int b0 = tid & ~31, j = 0; b0 < a.B; b0 += nthreads, ++j) {
    const int b = b0 + (tid & 31);
    const int g = b < a.B ? group_of(b) : -1;
    const int L = b < a.B ? length(b, j, true) : 0;
    const bool in = takes_part(L, g) && b < a.B;
    const int start = start_of(L);
    tails += (L + kTile - 1) / kTile - start / kTile;
    if (in && start > 0) atomicMax(&s_lo[g], (start + kTile - 1) / kTile * kTile);
    const unsigned votes = __ballot_sync(kFull, in);
    const int g_first = __shfl_sync(kFull, g, votes ? __ffs(votes) - 1 : 0);
    if (__all_sync(kFull, !in || g == g_first)) {
      if (in && (tid & 31) == __ffs(votes) - 1) {
        atomicAdd(&s_in[g], __popc(votes));
        atomicMin(&s_first[g], b);
        atomicMax(&s_last[g], b0 + 31 - __clz(votes));
      }
    } else if (in) {
      atomicAdd(&s_in[g], 1);
      atomicMin(&s_first[g], b);
      atomicMax(&s_last[g], b);
    }
  }
  tails = __reduce_add_sync(kFull, tails);
  if ((tid & 31) == 0) atomicAdd(&s_tails, tails);
  __syncthreads();

  int early = 0;  // thread 0: CTAs of the decode kernel that find an SM free
  // units, flat tiles, slots
  const int up_max = a.unit_rows / a.G;
  if (mine) {
    int run = 0;
    for (int g0 = 0; g0 < a.NG; g0 += step) {
      const int g = g0 + tid;
      int x = 0;
      if (g < a.NG) {
        // Units are cut over the rows from the first that takes part to the last
        // (idle rows are mostly the end of a padded batch). Each reads the prefix
        // once, as a sequence by itself does, so there must be fewer of them than
        // rows that take part.
        const int n = max(s_last[g] - s_first[g] + 1, 0);
        Units u;
        u.nut = n <= up_max ? (n > 0) : (n + up_max - 1) / up_max;
        if (s_in[g] <= u.nut || s_lo[g] >= s_pre[g]) s_pre[g] = s_lo[g] = 0;
        const int span = s_pre[g] - s_lo[g];
        if (span > 0) atomicSub(&s_tails, s_in[g] * (span / kTile));
        u.nt = (span + a.kv - 1) / a.kv;
        u.up = u.nut <= 1 ? n : (n + u.nut - 1) / u.nut;
        u.up_mul = u.nut <= 1 ? 0u : 0xffffffffu / static_cast<uint32_t>(max(u.up, 1)) + 1u;
        s_units[g] = u;
        x = a.Hkv * u.nut * u.nt;
        if (x > 0) atomicAdd(&s_nunits, a.Hkv * u.nut);
        if (a.halves && u.up * a.G > a.unit_rows / 2) atomicAdd(&s_dual, x);
      }
      const int y = scan<ONE>(x, 0, add, &total);
      if (g < a.NG) s_in[g] = run + y - x;
      run += total;
    }
    if constexpr (ONE) __syncwarp(); else __syncthreads();
    const int tiles = run;
    const int ctas = share_sms(a, tiles, s_dual, s_nunits, s_tails * a.Hkv);
    const int wsz = max((tiles + ctas - 1) / ctas, a.min_tiles);
    if (tid == 0) {
      s_tiles = tiles;
      s_wsz = wsz;
      a.plan[kShWsz] = wsz;
      // the prefix kernel's CTAs with work; the others leave their SMs at once, to
      // the first CTAs of the decode kernel
      const int busy = (tiles + wsz - 1) / wsz;
      early = busy > a.whole ? a.decode_ctas
                             : max(1, min(a.decode_ctas, (a.ctas - busy) * a.decode_per_sm));
    }
    run = 0;
    for (int g0 = 0; g0 < a.NG; g0 += step) {
      const int g = g0 + tid;
      int x = 0;
      if (g < a.NG) {
        const Units u = s_units[g];
        const int first = s_in[g], last = first + a.Hkv * u.nut * u.nt - 1;
        const int w0 = first / wsz;
        s_w0[g] = w0;
        if (u.nt > 0) x = (a.Hkv * u.nut + last / wsz - w0) * u.up;
      }
      const int y = scan<ONE>(x, 0, add, &total);
      if (g < a.NG) s_base[g] = run + y - x;
      run += total;
    }
  }
  __syncthreads();
  const int wsz = s_wsz, tiles = s_tiles;
  auto record = [&](int g) -> SharedGroup {
    SharedGroup r = {};
    if (g >= a.NG) return r;
    const Units u = s_units[g];
    r.r0 = r.table_row = s_first[g];
    r.n = max(s_last[g] - s_first[g] + 1, 0);
    r.prefix = s_pre[g] - s_lo[g];
    r.first = s_lo[g];
    r.f0 = s_in[g];
    r.nt = u.nt;
    r.nut = u.nut;
    r.up = u.up;
    r.base = s_base[g];
    r.dual = a.halves && u.up * a.G > a.unit_rows / 2;
    r.wfirst = s_w0[g];
    return r;
  };
  SharedGroup* groups = const_cast<SharedGroup*>(shared_groups(a.plan, a.ctas));
  for (int g = tid; g < a.NG; g += nthreads) groups[g] = record(g);
  SharedCta* ctas = const_cast<SharedCta*>(shared_ctas(a.plan));
  for (int w = tid; w < a.ctas; w += nthreads) {
    SharedCta c;
    c.f0 = static_cast<int>(min(static_cast<long long>(w) * wsz, static_cast<long long>(tiles)));
    c.f1 = min(c.f0 + wsz, tiles);
    // the last group that starts at or before f0: those without tiles share
    // their start with the next one
    int lo = 0, hi = a.NG;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_in[mid] <= c.f0) lo = mid; else hi = mid;
    }
    c.group = lo;
    c.pad = 0;
    c.g = record(lo);
    ctas[w] = c;
  }
  SharedRow* rows = const_cast<SharedRow*>(shared_rows(a.plan, a.ctas, a.NG));
  int before = 0, some = 0;  // units of the rows of earlier rounds, rows with any
  for (int b0 = 0, j = 0; b0 < a.B; b0 += nthreads, ++j) {
    const int b = b0 + tid;
    const int g = b < a.B ? group_of(b) : -1;
    const int L = b < a.B ? length(b, j) : 0;
    SharedRow r = {};
    r.start = start_of(L);
    r.len = L;
    r.tiles = (L + kTile - 1) / kTile - r.start / kTile;
    if (takes_part(L, g)) {
      const Units u = s_units[g];
      const int i = b - s_first[g];
      const int ut = u.up_mul ? (u.up == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), u.up_mul))) : 0;
      r.head = s_lo[g] / kTile - r.start / kTile;
      r.tiles -= (s_pre[g] - s_lo[g]) / kTile;
      r.nt = u.nt;
      r.f0 = s_in[g] + ut * u.nt;
      r.kv_step = u.nut * u.nt;
      r.slot0 = s_base[g] + i - ut * u.up;
      r.lid0 = ut - s_w0[g];
      r.up = u.up;
      r.nut = u.nut;
    }
    int all;
    const int units = r.tiles > 0 ? r.tiles + 1 : 0;
    r.pref = before + scan<false>(units, 0, add, &all) - units;
    before += all;
    some += __syncthreads_count(units > 0);
    if (b < a.B) rows[b] = r;
  }
  if (tid == 0) {
    const unsigned warps = static_cast<unsigned>(early) * a.decode_warps;
    a.plan[kShTails] = before;
    // (A unit alone may be no tile. Pairs of two tiles whose partials are large, 8 KB
    // and more, are better left whole than joined from two warps: 95 rows of 64/8
    // heads of 256, 64.2 against 68.9 us. Smaller ones are not: 26 rows of 64/8 heads
    // of 128 with tails of up to 95 tokens 42.1 whole, 39.8 cut.)
    const int pair = a.wide_partials ? min((before + max(some, 1) - 1) / max(some, 1), 3) : 2;
    a.plan[kShTailsWs] = max(static_cast<int>((static_cast<unsigned>(before * a.Hkv) + warps - 1u) / warps),
                             max(a.decode_min_tiles, max(pair, 2)));
  }
  griddep_wait();  // what follows this kernel follows its predecessors too
}

}  // namespace

cudaError_t shared_plan_launch(const SharedPlanArgs& a, cudaStream_t s, bool pdl) {
  const size_t smem = (12 * static_cast<size_t>(a.NG) + 1) * sizeof(int);
  if (smem > 40 * 1024) {
    // Without asking, a CTA has 48 KB, its static arrays (0.3 KB) among them. (One
    // value, whichever thread sets it.)
    const cudaError_t e =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(shared_plan_kernel<false>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (12 * kMostGroups + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  const bool one = a.NG < 32;
  cfg.blockDim = dim3(a.B <= 1024 && one ? 256 : kMaxThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return one ? cudaLaunchKernelEx(&cfg, shared_plan_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, shared_plan_kernel<false>, a);
}

}  // namespace pa
