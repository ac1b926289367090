// Attention of a group's sequences over the prefix they share, on the
// 5th-generation tensor cores: one pass over the prefix's K/V for all of them.
//
// The queries of the n sequences of a group, G heads of one KV head each, are
// the rows of one matrix Q [n G x D]; every row attends to all of [0, P), so
//   S = Q K^T,  P = 2^(S c - m),  O += P V,  l += sum P
// with a running reference m per row, and no mask but the end of the last
// tile. Partials (O, m, l) go to workspace slots in the decode partials'
// layout, where the merge joins them with each sequence's own tail.
//
// Read once for all rows, the prefix costs 4 n G D operations a token and KV
// head for 4 D bytes (16-bit): memory-bound below about n G = 280 rows, tensor
// and exponential above. The flat space of K/V tiles is split evenly over one
// CTA per SM (shared_plan.cuh), whatever the groups' sizes.
//
// Roles as in the chunk kernel: a producer warp streams K and V tiles of kKv
// tokens through two-stage rings (TMA through the block table of one of the
// group's sequences), an MMA warp issues every product, and groups of four
// softmax warps serve one 128-row tile each (one row a thread). With two
// groups, a unit of more than 128 rows gives each group half of the rows on
// every tile; a smaller one gives both groups the same rows on every other
// tile, so that the tensor core always works for one group while the other
// is in its softmax. Per tile and group x:
//   S_x = Q_x K^T -> TMEM; P_x (16-bit, packed in pairs) over the first half of
//   each 64 columns of S_x; O_x += P_x V from TMEM
// as in the chunk kernel, with its lazy reference max. K/V rows behind the
// prefix in its last tile are not loaded; their scores are masked and their V
// rows zeroed in shared memory. head_dim 256 takes one group and 64-token
// tiles (its O fills half of the tensor memory, its Q 64 KB).
//
// FP8 caches: two converter warps turn each raw e4m3 tile into the f16 tile the
// products read (exact); Q is rescaled per row by a power of two to f16's
// range, which the row's score scale undoes.
#include "attn_tc.cuh"
#include "pa_internal.h"
#include "ptx.cuh"
#include "shared_plan.cuh"
#include "step_ops.h"
#include "tc.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;
constexpr int kGroupThreads = 128;
constexpr int kConvWarps = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;  // bound of every wait (2 s)
constexpr float kFloor = -1e30f;             // reference-max start
constexpr float kRescaleAbove = 8.f;         // log2 units
constexpr unsigned kFull = 0xffffffffu;

// barriers: K and V rings (full, empty; two stages each); per group x: S_x
// computed, P_x written, O_x product complete, Q_x staged; FP8: converted K
// written / read, converted V (two buffers) written / read
constexpr int kBarKFull = 0, kBarKEmpty = 2, kBarVFull = 4, kBarVEmpty = 6, kBarS = 8, kBarP = 10,
              kBarO = 12, kBarQ = 14, kBarCKFull = 16, kBarCKFree = 17, kBarCVFull = 18,
              kBarCVFree = 20, kNumBars = 22;

template <int D, bool FP8>
struct Cfg {
  static constexpr int kGroups = D == 256 ? 1 : 2;  // softmax groups
  static constexpr int kKv = D == 256 ? 64 : 128;   // tokens a tile
  static constexpr int kSlices = kKv / 16;
  static constexpr int kBoxes = D / 64;  // 64-dim boxes of a 16-bit tile
  static constexpr int kMmaWarp = 4 * kGroups, kLoadWarp = kMmaWarp + 1, kConvWarp0 = kLoadWarp + 1;
  static constexpr int kThreads = (kConvWarp0 + (FP8 ? kConvWarps : 0)) * 32;
  static constexpr uint32_t kQBox = kRows * 128, kQBytes = kBoxes * kQBox;  // one group's Q
  static constexpr uint32_t kBox = kKv * 128, kTile = kBoxes * kBox;        // 16-bit K or V tile
  static constexpr uint32_t kRawBoxes = FP8 ? D / 128 : kBoxes;             // 128-byte boxes
  static constexpr uint32_t kRing = kRawBoxes * kBox;                       // ring tile
  static constexpr uint32_t kQ = 0, kK = kQ + kGroups * kQBytes, kV = kK + 2 * kRing;
  static constexpr uint32_t kKc = kV + 2 * kRing, kVc = kKc + (FP8 ? kTile : 0);
  static constexpr uint32_t kBar = kVc + (FP8 ? 2 * kTile : 0);
  static constexpr uint32_t kSlot = kBar + 8 * kNumBars;
  static constexpr uint32_t kBytes = kSlot + 16 + 1024;  // + room to align the base to 1 KB
  static constexpr uint32_t kColS = 0, kColO = kGroups * kKv;
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
  static_assert(kColO + kGroups * D <= kTmemCols, "tensor memory");
};

__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait_bounded(bar, parity, kWaitNs));
}

// One run of this CTA's tiles inside one unit.
struct Segment {
  SharedGroup g;
  int kvh, ut;
  int b0, np;  // first sequence and number of pairs
  int t0, nt;  // tiles [t0, t0 + nt) of the prefix
  bool dual;   // each group has its own rows (else its own tiles)
  int slot0;   // slot of x 0, pair 0
};

// The segment that starts at flat tile f (gi: the group found last, or -1).
__device__ __forceinline__ void segment_at(const PrefixArgs& a, int f, int f_end, int* gi,
                                           Segment* s) {
  const SharedGroup* groups = shared_groups(a.plan);
  if (*gi < 0) {  // the last group with f0 <= f (those without tiles come before)
    int lo = 0, hi = a.NG;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (groups[mid].f0 <= f) lo = mid; else hi = mid;
    }
    *gi = lo;
    s->g = groups[lo];
  }
  while (f >= s->g.f0 + a.Hkv * s->g.nut * s->g.nt && *gi + 1 < a.NG) s->g = groups[++*gi];
  const int rem = f - s->g.f0, unit = rem / s->g.nt;
  s->t0 = rem - unit * s->g.nt;
  s->nt = min(s->g.nt - s->t0, f_end - f);
  s->kvh = unit / s->g.nut;
  s->ut = unit - s->kvh * s->g.nut;
  s->b0 = s->g.r0 + s->ut * s->g.up;
  s->np = min(s->g.up, s->g.n - s->ut * s->g.up);
  s->dual = s->g.sub == 1;
  s->slot0 = s->g.base + (unit + static_cast<int>(blockIdx.x) - s->g.wfirst) * s->g.sub * s->g.up;
}

template <int QT, int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    prefix_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PrefixArgs a) {
  using C = Cfg<D, FP8>;
  constexpr bool kBf16 = !FP8 && QT == kBF16;  // operand type of the products
  constexpr int NX = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base + C::kQ, sK = base + C::kK, sV = base + C::kV;
  const uint32_t sKc = base + C::kKc, sVc = base + C::kVc;
  auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * i; };
  const uint32_t* tslot = reinterpret_cast<const uint32_t*>(smem_raw + (base - raw) + C::kSlot);
  // the 16-bit K and V tiles the products read for this CTA's c-th tile, and
  // the barrier (with parity) that says they are ready
  auto tile_k = [&](int c) -> uint32_t { return FP8 ? sKc : sK + (c & 1) * C::kTile; };
  auto tile_v = [&](int c) -> uint32_t { return (FP8 ? sVc : sV) + (c & 1) * C::kTile; };
  auto k_ready = [&](int c) -> uint32_t { return FP8 ? bar(kBarCKFull) : bar(kBarKFull + (c & 1)); };
  auto v_ready = [&](int c) -> uint32_t { return bar((FP8 ? kBarCVFull : kBarVFull) + (c & 1)); };
  auto k_par = [&](int c) -> uint32_t { return FP8 ? c & 1 : (c >> 1) & 1; };
  auto v_par = [&](int c) -> uint32_t { return (c >> 1) & 1; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), FP8 ? kConvWarps * 32 : 1);
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarVEmpty + i), FP8 ? kConvWarps * 32 : 1);
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), kGroupThreads);
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarQ + i), kGroupThreads);
      mbar_init(bar(kBarCVFull + i), kConvWarps * 32);
      mbar_init(bar(kBarCVFree + i), 1);
    }
    mbar_init(bar(kBarCKFull), kConvWarps * 32);
    mbar_init(bar(kBarCKFree), 1);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(base + C::kSlot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  griddep_wait();  // the plan, and behind it the caches and queries, are written
  griddep_launch_dependents();

  const int total = a.plan[kShTotal], wsz = a.plan[kShWsz];
  const int f0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * wsz, static_cast<long long>(total)));
  const int f1 = min(f0 + wsz, total);
  const int ntiles = f1 - f0;  // of this CTA, over all its segments
  int gi = -1;
  Segment sg;

  if (warp == C::kLoadWarp) {
    // ------------------------------------------------------------ producer
    // K (or V) tile: lanes 0..kSlices-1 each look up one 16-token slice in the
    // block table and copy its 128-byte boxes; slices behind the prefix are
    // not loaded
    auto load = [&](int c, int t, bool is_v) {
      const uint32_t full = bar((is_v ? kBarVFull : kBarKFull) + (c & 1));
      const int pos0 = t * C::kKv + 16 * lane;
      int row = -1;
      if (lane < C::kSlices && pos0 < sg.g.prefix) {
        int blk = __ldg(a.block_tables + static_cast<size_t>(sg.g.table_row) * a.MB + pos0 / a.bs);
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.NB)) {
          atomicOr(a.err, PA_DEVERR_BLOCK_ID);
          blk = 0;
        }
        row = (blk * a.Hkv + sg.kvh) * a.bs + pos0 % a.bs;
      }
      const int nslices = __popc(__ballot_sync(kFull, row >= 0));
      if (lane == 0) mbar_arrive_expect_tx(full, nslices * C::kRawBoxes * 2048);
      __syncwarp();
      if (row >= 0) {
        const uint32_t dst = (is_v ? sV : sK) + (c & 1) * C::kRing + lane * 2048;
#pragma unroll
        for (int box = 0; box < static_cast<int>(C::kRawBoxes); ++box)
          tma_load_2d(dst + box * C::kBox, is_v ? &tmV : &tmK, box * (FP8 ? 128 : 64), row, full);
      }
      __syncwarp();
    };
    bool ok = true;
    int c = 0;
    for (int f = f0; ok && f < f1; f += sg.nt) {
      segment_at(a, f, f1, &gi, &sg);
      for (int n = 0; ok && n < sg.nt; ++n, ++c) {
        const uint32_t par = ((c - 2) >> 1) & 1;  // release of the stage's last tile
        if (c >= 2 && !(ok = wait_all(bar(kBarKEmpty + (c & 1)), par))) break;
        load(c, sg.t0 + n, false);
        if (c >= 2 && !(ok = wait_all(bar(kBarVEmpty + (c & 1)), par))) break;
        load(c, sg.t0 + n, true);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issue
    constexpr uint32_t idS = tc::idesc_f16(kRows, C::kKv, kBf16, false);
    constexpr uint32_t idO = tc::idesc_f16(kRows, D, kBf16, true);
    auto issue_s = [&](int x, int c) {
      if (lane == 0) {
        const uint64_t dQ = tc::sdesc_sw128(sQ + x * C::kQBytes, 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(tile_k(c), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc::mma_f16(tmem + C::kColS + C::kKv * x,
                      dQ + (((ks >> 2) * C::kQBox + (ks & 3) * 32) >> 4),
                      dK + (((ks >> 2) * C::kBox + (ks & 3) * 32) >> 4), idS, ks > 0);
        tc::commit(bar(kBarS + x));
      }
      __syncwarp();
    };
    // O_x (+)= P_x V: 16 tokens a step, P in 8 columns each from 64 h on
    auto issue_o = [&](int x, int c, bool first) {
      if (lane == 0) {
        const uint64_t dV = tc::sdesc_sw128(tile_v(c), C::kBox, 1024);
#pragma unroll
        for (int k = 0; k < C::kKv / 16; ++k)
          tc::mma_f16_ta(tmem + C::kColO + D * x,
                         tmem + C::kColS + C::kKv * x + 64 * (k >> 2) + 8 * (k & 3),
                         dV + 128 * k, idO, !first || k > 0);
        tc::commit(bar(kBarO + x));
      }
      __syncwarp();
    };
    // A release is committed only when something will wait for it, so no
    // arrive outlives the CTA.
    auto release_k = [&](int c) {
      if (lane == 0) {
        if (FP8 && c + 1 < ntiles) tc::commit(bar(kBarCKFree));
        if (!FP8 && c + 2 < ntiles) tc::commit(bar(kBarKEmpty + (c & 1)));
      }
      __syncwarp();
    };
    auto release_v = [&](int c) {
      if (lane == 0 && c + 2 < ntiles) tc::commit(bar((FP8 ? kBarCVFree : kBarVEmpty) + (c & 1)));
      __syncwarp();
    };
    bool ok = true;
    int c0 = 0;
    int ops[2] = {0, 0};   // products O_x issued so far
    int segs[2] = {0, 0};  // segments of each group so far (those it has tiles of)
    for (int f = f0; ok && f < f1; f += sg.nt, c0 += sg.nt) {
      segment_at(a, f, f1, &gi, &sg);
      // the i-th S (and O) product of the segment: group i % NX, tile i / NX
      // (its own rows) or i (its own tiles)
      const bool dual = NX == 2 && sg.dual;
      const int nops = dual ? 2 * sg.nt : sg.nt;
      auto x_of = [&](int i) -> int { return NX == 2 ? i & 1 : 0; };
      auto c_of = [&](int i) -> int { return c0 + (dual ? i >> 1 : i); };
      auto first_use = [&](int i) -> bool { return !dual || !(i & 1); };
      auto last_use = [&](int i) -> bool { return !dual || (i & 1); };
      for (int i = 0; i < NX && i < nops; ++i) {
        if (!(ok = wait_all(bar(kBarQ + i), segs[i]++ & 1))) break;
        if (first_use(i) && !(ok = wait_all(k_ready(c_of(i)), k_par(c_of(i))))) break;
        tc::fence_after_sync();
        issue_s(x_of(i), c_of(i));
        if (last_use(i)) release_k(c_of(i));
      }
      for (int i = 0; ok && i < nops; ++i) {
        const int x = x_of(i), c = c_of(i);
        const uint32_t par = ops[x] & 1;
        if (!(ok = wait_all(bar(kBarP + x), par))) break;  // P_x (and clean V rows) written
        if (first_use(i) && !(ok = wait_all(v_ready(c), v_par(c)))) break;
        tc::fence_after_sync();
        issue_o(x, c, i < NX);
        ++ops[x];
        if (last_use(i)) release_v(c);
        if (i + NX < nops) {
          const int cn = c_of(i + NX);
          if (first_use(i + NX) && !(ok = wait_all(k_ready(cn), k_par(cn)))) break;
          if (!(ok = wait_all(bar(kBarO + x), par))) break;  // P_x consumed
          tc::fence_after_sync();
          issue_s(x, cn);
          if (last_use(i + NX)) release_k(cn);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  } else if (warp >= C::kConvWarp0) {
    // ------------------------------------------------------------ FP8 converters
    // e4m3 tile c, ring stage c & 1 -> the f16 buffer: a 16-byte chunk of 16
    // codes becomes two 16-byte chunks of f16 in the 64-dim box that holds
    // them; V rows behind the prefix are written as zeros.
    if constexpr (FP8) {
      constexpr int kChunks = D / 16, kPer = kConvWarps * 32 / kChunks;
      const int ct = tid - C::kConvWarp0 * 32;
      const int ch = ct % kChunks, q0 = ct / kChunks;
      bool ok = true;
      int c = 0;
      for (int f = f0; ok && f < f1; f += sg.nt) {
        segment_at(a, f, f1, &gi, &sg);
        for (int n = 0; ok && n < sg.nt; ++n, ++c) {
          const int lim = sg.g.prefix - (sg.t0 + n) * C::kKv;  // rows of the tile inside the prefix
          for (int is_v = 0; is_v < 2; ++is_v) {
            if (!(ok = wait_all(bar((is_v ? kBarVFull : kBarKFull) + (c & 1)), (c >> 1) & 1))) break;
            if (!is_v && c > 0 && !(ok = wait_all(bar(kBarCKFree), (c - 1) & 1))) break;
            if (is_v && c > 1 && !(ok = wait_all(bar(kBarCVFree + (c & 1)), ((c - 2) >> 1) & 1))) break;
            const uint32_t src = (is_v ? sV : sK) + (c & 1) * C::kRing + (ch >> 3) * C::kBox;
            const uint32_t dst = (is_v ? sVc + (c & 1) * C::kTile : sKc) + (ch >> 2) * C::kBox;
            const int c16 = 2 * (ch & 3);
#pragma unroll 8
            for (int k = 0; k < C::kKv / kPer; ++k) {
              const int r = q0 + kPer * k;
              uint32_t w[4];
              lds_v4(src + r * 128 + (((ch & 7) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
              uint32_t h[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                h[2 * i] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] & 0xffffu));
                h[2 * i + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16));
              }
              const bool zero = is_v && r >= lim;
              sts_v4(dst + r * 128 + ((c16 ^ (r & 7)) << 4),
                     zero ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(h[0], h[1], h[2], h[3]));
              sts_v4(dst + r * 128 + (((c16 + 1) ^ (r & 7)) << 4),
                     zero ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(h[4], h[5], h[6], h[7]));
            }
            fence_proxy_async();  // the f16 tile, visible to the tensor core
            mbar_arrive(bar(is_v ? kBarCVFull + (c & 1) : kBarCKFull));
            // reload the stage (where something will wait for it)
            mbar_arrive(bar((is_v ? kBarVEmpty : kBarKEmpty) + (c & 1)));
          }
        }
      }
      if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;           // group
    const int r = tid - x * kRows;     // row of the tile = tensor-memory lane
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = trow + C::kColS + C::kKv * x, tO = trow + C::kColO + D * x;
    const SharedRow* rows = shared_rows(a.plan, a.NG);
    bool ok = true;
    int c0 = 0, op = 0;  // products of this group so far
    for (int f = f0; ok && f < f1; f += sg.nt, c0 += sg.nt) {
      segment_at(a, f, f1, &gi, &sg);
      const bool dual = NX == 2 && sg.dual;
      const int nj = dual || NX == 1 ? sg.nt : (sg.nt - x + 1) >> 1;  // this group's tiles
      const int row = r + (dual ? x * kRows : 0);  // row of the unit: pair * G + head
      const int pair = row / a.G, h = row - pair * a.G;
      const int b = sg.b0 + pair;
      // rows of the last pairs, and of sequences that take no part, stay zero
      const bool valid = pair < sg.np && rows[b].nt > 0;
      float sc = fabsf(a.score_scale);
      // A group without tiles in a segment (the second half of a single tile)
      // stages no Q: with nothing to wait for it would run ahead of the barrier.
      if (nj > 0) {  // Q row -> shared memory (K-major, 128-byte swizzle)
        const uint32_t flip = a.score_scale < 0.f ? 0x80008000u : 0u;
        const size_t qrow =
            (static_cast<size_t>(valid ? b : 0) * a.Hq + static_cast<size_t>(sg.kvh) * a.G + h) * D;
        const uint4* src =
            reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) + qrow);
        const uint32_t dst = sQ + x * C::kQBytes + r * 128;
        auto f32 = [&](uint32_t w, int hi) -> float {
          const uint16_t v = static_cast<uint16_t>(hi ? w >> 16 : w & 0xffffu);
          return QT == kBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16)
                             : __half2float(__ushort_as_half(v));
        };
        int sh = 0;
        if constexpr (FP8) {
          // f16 after a power-of-two rescale: largest magnitude in [2^14, 2^15)
          float amax = 0.f;
#pragma unroll
          for (int ch = 0; ch < D / 8; ++ch) {
            const uint4 v = valid ? src[ch] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f32(w4[i >> 1], i & 1)));
          }
          if (amax > 0.f && amax < INFINITY) {
            int e;
            frexpf(amax, &e);
            sh = e - 15;
          }
          sc = ldexpf(sc, sh);
        }
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch) {
          uint4 v = valid ? src[ch] : make_uint4(0u, 0u, 0u, 0u);
          if constexpr (FP8) {
            const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
            uint32_t o4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o4[i] = pack16x2<false>(ldexpf(f32(w4[i], 0), -sh), ldexpf(f32(w4[i], 1), -sh));
            v = make_uint4(o4[0], o4[1], o4[2], o4[3]);
          }
          v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
          sts_v4(dst + (ch >> 3) * C::kQBox + (((ch & 7) ^ (r & 7)) << 4), v);
        }
        fence_proxy_async();
        tc::fence_before_sync();  // the last segment's O has been read
        mbar_arrive(bar(kBarQ + x));
      }
      float ms = kFloor, l = 0.f;  // reference max (scaled, log2 units) and running sum
      for (int j = 0; j < nj; ++j, ++op) {
        const int n = dual || NX == 1 ? j : 2 * j + x;
        const int lim = min(sg.g.prefix - (sg.t0 + n) * C::kKv, C::kKv);  // tokens of the tile
        if (!(ok = wait_all(bar(kBarS + x), op & 1))) break;
        tc::fence_after_sync();
        const bool all_in = lim == C::kKv;
        uint32_t sv[2][32];
        float mxp[8];  // eight independent partial maxima (raw scores)
#pragma unroll
        for (int i = 0; i < 8; ++i) mxp[i] = -INFINITY;
#pragma unroll 1
        for (int hf = 0; hf < C::kKv / 64; ++hf) {
          tc::ld32_async(tS + 64 * hf, sv[0]);
          tc::ld32_async(tS + 64 * hf + 32, sv[1]);
          tc::wait_ld(sv[0], sv[1]);
          if (all_in) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              mxp[i & 7] = fmax3(mxp[i & 7], __uint_as_float(sv[i >> 4][(2 * i) & 31]),
                                 __uint_as_float(sv[i >> 4][(2 * i + 1) & 31]));
          } else {  // lim is even
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const bool in = 64 * hf + 2 * i < lim;
              mxp[i & 7] = fmax3(mxp[i & 7],
                                 in ? __uint_as_float(sv[i >> 4][(2 * i) & 31]) : -INFINITY,
                                 in ? __uint_as_float(sv[i >> 4][(2 * i + 1) & 31]) : -INFINITY);
            }
          }
        }
        const float mxr = fmaxf(fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])),
                                fmaxf(fmaxf(mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7])));
        const float mx = fmaxf(mxr * sc, kFloor);
        const bool grow = mx > ms + kRescaleAbove;
        if (j == 0) {
          ms = mx;  // nothing accumulated yet
        } else if (__any_sync(kFull, grow)) {
          // O_x is complete up to the last tile: S_x was issued after its product
          const float alpha = grow ? ex2(ms - mx) : 1.f;
#pragma unroll 1
          for (int d0 = 0; d0 < D; d0 += 32) {
            uint32_t ov[32];
            tc::ld32_async(tO + d0, ov);
            tc::wait_ld(ov);
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 o = __fmul2_rn(score_pair(ov, i), a2);
              ov[i] = __float_as_uint(o.x);
              ov[i + 1] = __float_as_uint(o.y);
            }
            tc::st32(tO + d0, ov);
          }
          l *= alpha;
          if (grow) ms = mx;
        }
        // P = 2^(s * sc - ms), packed in pairs over the columns of the scores
        // just used; the last half is still in registers
        const float2 sc2 = make_float2(sc, sc), nms2 = make_float2(-ms, -ms);
        float2 sp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sp[i] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int hf = C::kKv / 64 - 1; hf >= 0; --hf) {
          if (hf != C::kKv / 64 - 1) {
            tc::ld32_async(tS + 64 * hf, sv[0]);
            tc::ld32_async(tS + 64 * hf + 32, sv[1]);
            tc::wait_ld(sv[0], sv[1]);
          }
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float2 t = __ffma2_rn(score_pair(sv[i >> 4], (2 * i) & 31), sc2, nms2);
            float p0 = ex2(t.x), p1 = ex2(t.y);
            if (!all_in && 64 * hf + 2 * i >= lim) p0 = p1 = 0.f;
            sp[i & 3] = __fadd2_rn(sp[i & 3], make_float2(p0, p1));
            pk[i] = pack16x2<kBf16>(p0, p1);
          }
          tc::st32(tS + 64 * hf, pk);
        }
        const float2 s01 = __fadd2_rn(sp[0], sp[1]), s23 = __fadd2_rn(sp[2], sp[3]);
        const float2 st = __fadd2_rn(s01, s23);
        l += st.x + st.y;
        if (!FP8 && !all_in && !(dual && x == 1)) {
          // the prefix ends inside this tile: zero its V rows behind it once
          // the others have landed
          const int c = c0 + n;
          if (!(ok = wait_all(bar(kBarVFull + (c & 1)), (c >> 1) & 1))) break;
          const uint32_t vt = sV + (c & 1) * C::kTile;
          for (int i = lim * 8 + r; i < C::kKv * 8; i += kRows)
#pragma unroll
            for (int box = 0; box < C::kBoxes; ++box)
              sts_v4(vt + box * C::kBox + i * 16, make_uint4(0u, 0u, 0u, 0u));
          fence_proxy_async();
        }
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kBarP + x));
      }
      // the partial of this row: O as it is, its reference max and sum
      if (ok && nj > 0) ok = wait_all(bar(kBarO + x), (op - 1) & 1);
      tc::fence_after_sync();
      const bool some = ok && nj > 0;
      const int slot = sg.slot0 + (dual || NX == 1 ? 0 : x * sg.g.up) + pair;
      float* P = a.part + static_cast<size_t>(slot) * part_stride(a.G, D);
      const uint64_t keep = l2_evict_last();  // the merge reads them soon
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t ov[32];
        if (nj > 0) {
          tc::ld32_async(tO + d0, ov);
          tc::wait_ld(ov);
        }
        if (valid) {
          const float vs = some ? a.v_scale : 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float* o = reinterpret_cast<const float*>(ov) + i;
            const float4 v = some ? make_float4(o[0] * vs, o[1] * vs, o[2] * vs, o[3] * vs)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            st_f32x4_hint(P + h * D + d0 + i, v, keep);
          }
        }
      }
      if (valid) {
        st_f32_hint(P + a.G * D + h, some ? ms : kFloor, keep);
        st_f32_hint(P + a.G * D + a.G + h, some ? l : 0.f, keep);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  }

  // every MMA has completed (each group waited for its last product)
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int QT, int D, bool FP8>
cudaError_t launch_typed(const CUtensorMap& tk, const CUtensorMap& tv, const PrefixArgs& a,
                         int grid, cudaStream_t s, bool pdl) {
  // a function attribute of the current device's context: set every time, a
  // host-side store
  cudaError_t e = cudaFuncSetAttribute(prefix_attn_tc_kernel<QT, D, FP8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Cfg<D, FP8>::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg<D, FP8>::kThreads);
  cfg.dynamicSmemBytes = Cfg<D, FP8>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_attn_tc_kernel<QT, D, FP8>, tk, tv, a);
}

template <int QT>
cudaError_t launch_dim(bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                       const PrefixArgs& a, int grid, cudaStream_t s, bool pdl) {
  if (fp8) {
    if (D == 128) return launch_typed<QT, 128, true>(tk, tv, a, grid, s, pdl);
    if (D == 256) return launch_typed<QT, 256, true>(tk, tv, a, grid, s, pdl);
    return cudaErrorInvalidValue;
  }
  if (D == 64) return launch_typed<QT, 64, false>(tk, tv, a, grid, s, pdl);
  if (D == 128) return launch_typed<QT, 128, false>(tk, tv, a, grid, s, pdl);
  if (D == 256) return launch_typed<QT, 256, false>(tk, tv, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace

PrefixShape prefix_shape(int D) {
  return D == 256 ? PrefixShape{Cfg<256, false>::kKv, kRows, false}
                  : PrefixShape{Cfg<128, false>::kKv, 2 * kRows, true};
}

cudaError_t prefix_launch(int qt, bool fp8, int D, const CUtensorMap& tk, const CUtensorMap& tv,
                          const PrefixArgs& a, int grid, cudaStream_t s, bool pdl) {
  return qt == kBF16 ? launch_dim<kBF16>(fp8, D, tk, tv, a, grid, s, pdl)
                     : launch_dim<kF16>(fp8, D, tk, tv, a, grid, s, pdl);
}

}  // namespace pa
