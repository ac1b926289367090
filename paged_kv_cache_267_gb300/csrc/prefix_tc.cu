// Attention of a group's sequences over the prefix they share, on the
// 5th-generation tensor cores: one pass over the prefix's K/V for all of them.
//
// The queries of the n sequences of a group, G heads of one KV head each, are
// the rows of one matrix Q [n G x D]; every row attends to all of the positions
// that the kernel covers (shared_plan.cuh), so
//   S = Q K^T,  P = 2^(S c - m),  O += P V,  l += sum P
// with a running reference m per row, and no mask but the end of the last
// tile. Partials (O, m, l) go to workspace slots in the decode partials'
// layout, where the merge joins them with each sequence's own tail.
//
// Read once for all rows, the prefix costs 4 n G D operations a token and KV
// head for 4 D bytes (16-bit): memory-bound below about n G = 280 rows, tensor
// and exponential above. The flat space of K/V tiles is split evenly over the
// CTAs (shared_plan.cuh), whatever the groups' sizes.
//
// Roles as in the chunk kernel: producers stream K and V tiles of kKv tokens
// through rings (TMA through the block table of one of the group's sequences;
// the next tile's block ids are looked up while the last one's copies are
// awaited), one thread issues every product, and groups of four softmax warps
// serve one 128-row tile each (one row a thread). With two groups, a unit of
// more than 128 rows gives each group half of the rows on every tile; a smaller
// one gives both groups the same rows on every other tile, so that the tensor
// core always works for one group while the other is in its softmax. Per tile
// and group x:
//   S_x = Q_x K^T -> TMEM; P_x (16-bit, packed in pairs) over the first half of
//   each 64 columns of S_x; O_x += P_x V from TMEM
// with a lazy reference max. K/V rows behind the prefix in its last tile are not
// loaded; their scores are masked and their V rows zeroed in shared memory.
// head_dim 256 takes one group and 64-token tiles (its O fills half of the
// tensor memory, its Q 64 KB).
//
// A CTA's tiles are few (its share of one prefix), so what it does once a
// segment counts as much as the loop: Q is loaded, and the partials stored, by
// whole warps along the rows (through the Q buffer, which is free once the
// last S is done), 128 bytes and more a row at once. One thread a row, 16
// bytes each, had cost about 6,000 and 5,000-9,700 cycles a segment of at most
// 100,000.
//
// FP8 caches: six converter warps, every sixth eight rows each, turn each raw e4m3
// tile into the f16 tile the products read (exact), in two buffers each for K
// and V, so that a tile is converted while the one before is multiplied; Q is
// rescaled per row by a power of two to f16's range, which the row's score scale
// undoes. With two converter warps they bound the loop (2.19 us a tile of 128
// tokens and two row tiles; now 1.89, bf16 1.73).
//
// bf16, 256 queries of 4 heads on 8 KV heads, between prefixes of 16384 and 65536
// tokens (75.8 and 216.1 us): 1.73 us a tile of one SM for 16.8 MFLOP, 1.47 PFLOP/s
// over the chip, 0.77 of the measured peak; bound by the softmax's exponentials
// and the products in turn. Shares of one prefix are short: of a 4096-token prompt
// a CTA has four tiles, and of its 14 us about seven are the queries' way in, the
// first tiles' latency and the partials' way out. head_dim 64 has half the bytes
// and products a tile for the same exponentials; head_dim 256, with one group and
// one S, runs S, softmax and O of a tile one after the other.
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
constexpr int kConv = 6;  // FP8 converter warps
// Registers a thread where 16 warps share the SM's: softmax warps, all others.
constexpr int kSoftmaxRegs = 168, kOtherRegs = 88;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;  // bound of every wait (2 s)
constexpr uint64_t kDrainNs = 200000000ull;  // and of those after one ran out
constexpr float kFloor = -1e30f;             // reference-max start
constexpr float kRescaleAbove = 8.f;         // log2 units
// f16 weights are 2^7 times as large against their reference: at most 2^15, and
// subnormal below 2^-21 of it instead of 2^-14. (55,000 tokens of weight 2^-19.5
// behind one of weight 1: 0.1% off without it, nothing with it.)
constexpr float kF16Lift = 7.f;              // log2 units
constexpr unsigned kFull = 0xffffffffu;

// barriers: K and V rings (full, empty; up to kMaxStages each); per group x: S_x
// computed, P_x written, O_x product complete; all rows' Q staged; both groups at
// a segment's end; FP8: converted K and V (two buffers each) written / read
constexpr int kMaxStages = 4;
constexpr int kBarKFull = 0, kBarKEmpty = kBarKFull + kMaxStages, kBarVFull = kBarKEmpty + kMaxStages,
              kBarVEmpty = kBarVFull + kMaxStages, kBarS = kBarVEmpty + kMaxStages,
              kBarP = kBarS + 2, kBarO = kBarP + 2, kBarQ = kBarO + 2, kBarEnd = kBarQ + 1, kBarCKFull = kBarEnd + 1,
              kBarCKFree = kBarCKFull + 2, kBarCVFull = kBarCKFree + 2, kBarCVFree = kBarCVFull + 2,
              kBarDrain = kBarCVFree + 2, kNumBars = kBarDrain + 1;

// Stage and phase of a ring position.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

template <int D, bool FP8>
struct Cfg {
  static constexpr int kGroups = D == 256 ? 1 : 2;  // softmax groups
  static constexpr int kKv = D == 256 ? 64 : 128;   // tokens a tile
  static constexpr int kSlices = kKv / 16;
  static constexpr int kBoxes = D / 64;  // 64-dim boxes of a 16-bit tile
  // 16-bit tiles are loaded by one warp for K and one for V: a V stage is held
  // through a softmax, a K stage only through its product, and in one warp K
  // loads would wait behind V's
  static constexpr int kLoadWarps = FP8 ? 1 : 2;
  static constexpr int kKStages = FP8 ? 1 : (D == 64 ? 4 : 2), kVStages = FP8 ? 1 : (D == 64 ? 4 : 3);
  static constexpr int kMmaWarp = 4 * kGroups, kLoadWarp = kMmaWarp + 1,
                       kConvWarp0 = kLoadWarp + kLoadWarps;
  static constexpr int kThreads = (kConvWarp0 + (FP8 ? kConv : 0)) * 32;
  // more than 12 warps leave each thread 128 registers, too few for the softmax:
  // its warps get what the others hand back
  static constexpr bool kSplitRegs = kThreads > 384;
  static_assert(!kSplitRegs || (kThreads == 512 && kGroups == 2 &&
                                kSoftmaxRegs + kOtherRegs == 2 * 128), "registers of the block");
  static constexpr uint32_t kQBox = kRows * 128, kQBytes = kBoxes * kQBox;  // one group's Q
  static constexpr uint32_t kBox = kKv * 128, kTile = kBoxes * kBox;        // 16-bit K or V tile
  static constexpr uint32_t kRawBoxes = FP8 ? D / 128 : kBoxes;             // 128-byte boxes
  static constexpr uint32_t kRing = kRawBoxes * kBox;                       // ring tile
  static constexpr uint32_t kQ = 0, kK = kQ + kGroups * kQBytes, kV = kK + kKStages * kRing;
  static constexpr uint32_t kKc = kV + kVStages * kRing, kVc = kKc + (FP8 ? 2 * kTile : 0);
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

// The segment that starts at flat tile f, in the group of s->g or one behind.
__device__ __forceinline__ void segment_at(const PrefixArgs& a, int f, int f_end, int* gi,
                                           Segment* s) {
  while (f >= s->g.f0 + a.Hkv * s->g.nut * s->g.nt && *gi + 1 < a.NG)
    s->g = shared_groups(a.plan, a.ctas)[++*gi];
  const int rem = f - s->g.f0, unit = rem < s->g.nt ? 0 : rem / s->g.nt;
  s->t0 = rem - unit * s->g.nt;
  s->nt = min(s->g.nt - s->t0, f_end - f);
  s->kvh = s->g.nut == 1 ? unit : unit / s->g.nut;
  s->ut = unit - s->kvh * s->g.nut;
  s->b0 = s->g.r0 + s->ut * s->g.up;
  s->np = min(s->g.up, s->g.n - s->ut * s->g.up);
  s->dual = s->g.dual != 0;
  s->slot0 = s->g.base + (unit + static_cast<int>(blockIdx.x) - s->g.wfirst) * s->g.up;
}

// Two 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void st2(uint32_t taddr, float a, float b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "f"(a), "f"(b)
               : "memory");
}
__device__ __forceinline__ float2 ld2(uint32_t taddr) {
  float a, b;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a), "=f"(b)
      : "r"(taddr)
      : "memory");
  return make_float2(a, b);
}

template <int QT>
__device__ __forceinline__ float f32_of(uint32_t w, int hi) {
  const uint16_t v = static_cast<uint16_t>(hi ? w >> 16 : w & 0xffffu);
  return QT == kBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16)
                     : __half2float(__ushort_as_half(v));
}

template <int QT, int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1)
    prefix_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const PrefixArgs a) {
  using C = Cfg<D, FP8>;
  constexpr bool kBf16 = !FP8 && QT == kBF16;  // operand type of the products
  constexpr float kLift = kBf16 ? 0.f : kF16Lift;
  constexpr int NX = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base + C::kQ, sK = base + C::kK, sV = base + C::kV;
  const uint32_t sKc = base + C::kKc, sVc = base + C::kVc;
  auto bar = [&](int i) -> uint32_t { return base + C::kBar + 8u * i; };
  const uint32_t* tslot = reinterpret_cast<const uint32_t*>(smem_raw + (base - raw) + C::kSlot);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), FP8 ? kConv * 32 : 1);
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarVEmpty + i), FP8 ? kConv * 32 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarS + i), 1);
      mbar_init(bar(kBarP + i), kGroupThreads);
      mbar_init(bar(kBarO + i), 1);
      mbar_init(bar(kBarCKFull + i), kConv * 32);
      mbar_init(bar(kBarCKFree + i), 1);
      mbar_init(bar(kBarCVFull + i), kConv * 32);
      mbar_init(bar(kBarCVFree + i), 1);
    }
    mbar_init(bar(kBarQ), NX * kGroupThreads);
    mbar_init(bar(kBarEnd), NX * kGroupThreads);
    mbar_init(bar(kBarDrain), 1);
    fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(base + C::kSlot, kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  griddep_wait();  // the plan, and behind it the caches and queries, are written
  griddep_launch_dependents();

  Segment sg;
  const SharedCta mine = shared_ctas(a.plan)[blockIdx.x];
  sg.g = mine.g;
  const int f0 = mine.f0, f1 = mine.f1;
  const int ntiles = f1 - f0;  // of this CTA, over all its segments
  int gi = mine.group;

  if (warp >= C::kMmaWarp) {
    if constexpr (C::kSplitRegs)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp >= C::kLoadWarp && warp < C::kConvWarp0) {
      // ------------------------------------------------------------ producers
      // Lanes 0..kSlices-1 each look up one 16-token slice of a tile in the block
      // table and copy its 128-byte boxes; slices behind the prefix (row < 0)
      // are not loaded.
      auto row_of = [&](int t) -> int {
        const int at = t * C::kKv + 16 * lane, pos0 = sg.g.first + at;
        if (lane >= C::kSlices || at >= sg.g.prefix) return -1;
        int blk = __ldg(a.block_tables + static_cast<size_t>(sg.g.table_row) * a.MB + pos0 / a.bs);
        if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.NB)) {
          atomicOr(a.err, PA_DEVERR_BLOCK_ID);
          blk = 0;
        }
        return (blk * a.Hkv + sg.kvh) * a.bs + pos0 % a.bs;
      };
      auto load = [&](int stage, int row, bool is_v) {
        const uint32_t full = bar((is_v ? kBarVFull : kBarKFull) + stage);
        const int nslices = __popc(__ballot_sync(kFull, row >= 0));
        if (lane == 0) mbar_arrive_expect_tx(full, nslices * C::kRawBoxes * 2048);
        __syncwarp();
        if (row >= 0) {
          const uint32_t dst = (is_v ? sV : sK) + stage * C::kRing + lane * 2048;
#pragma unroll
          for (int box = 0; box < static_cast<int>(C::kRawBoxes); ++box)
            tma_load_2d(dst + box * C::kBox, is_v ? &tmV : &tmK, box * (FP8 ? 128 : 64), row, full);
        }
        __syncwarp();
      };
      const bool do_k = C::kLoadWarps == 1 || warp == C::kLoadWarp;
      const bool do_v = C::kLoadWarps == 1 || warp != C::kLoadWarp;
      bool ok = true;
      Ring kr, vr;
      int c = 0, nk = 0, nv = 0;  // tiles so far; K and V loads
      for (int f = f0; ok && f < f1; f += sg.nt) {
        segment_at(a, f, f1, &gi, &sg);
        int row = row_of(sg.t0);
        for (int n = 0; ok && n < sg.nt; ++n, ++c) {
          // looked up while the waits below run
          const int next = n + 1 < sg.nt ? row_of(sg.t0 + n + 1) : -1;
          if (do_k) {  // the release of the stage's last tile: the phase before
            if (c >= C::kKStages && !(ok = wait_all(bar(kBarKEmpty + kr.stage), kr.phase ^ 1))) break;
            load(kr.stage, row, false);
            kr.next(C::kKStages);
            ++nk;
          }
          if (do_v) {
            if (c >= C::kVStages && !(ok = wait_all(bar(kBarVEmpty + vr.stage), vr.phase ^ 1))) break;
            load(vr.stage, row, true);
            vr.next(C::kVStages);
            ++nv;
          }
          row = next;
        }
      }
      if (!ok) {
        if (lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
        // no copy outlives the CTA
        for (int i = max(nk - C::kKStages, 0); i < nk; ++i)
          (void)mbar_wait_bounded(bar(kBarKFull + i % C::kKStages), (i / C::kKStages) & 1, kDrainNs);
        for (int i = max(nv - C::kVStages, 0); i < nv; ++i)
          (void)mbar_wait_bounded(bar(kBarVFull + i % C::kVStages), (i / C::kVStages) & 1, kDrainNs);
      }
    } else if (warp == C::kMmaWarp) {
      // ------------------------------------------------------------ MMA issue
      // One thread does all of it, and little besides: its own instructions are
      // on the critical path of every tile (a wait by the whole warp costs about
      // 150 cycles even when there is nothing to wait for, the products of one
      // tile and group about 1,200).
      if (lane == 0) {
        constexpr uint32_t idS = tc::idesc_f16(kRows, C::kKv, kBf16, false);
        constexpr uint32_t idO = tc::idesc_f16(kRows, D, kBf16, true);
        // Positions of the K and V tiles in use, and the barriers that say they
        // are ready: the ring's, or the converted buffers' (two of each).
        constexpr int KB = FP8 ? 2 : C::kKStages, VB = FP8 ? 2 : C::kVStages;
        constexpr int kKReady = FP8 ? kBarCKFull : kBarKFull, kKFree = FP8 ? kBarCKFree : kBarKEmpty;
        constexpr int kVReady = FP8 ? kBarCVFull : kBarVFull, kVFree = FP8 ? kBarCVFree : kBarVEmpty;
        const uint64_t dQ = tc::sdesc_sw128(sQ, 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(FP8 ? sKc : sK, 16, 1024);
        const uint64_t dV = tc::sdesc_sw128(FP8 ? sVc : sV, C::kBox, 1024);
        Ring kr, vr;
        // releases still to come: one is committed only when something will wait
        // for it, so that no arrive outlives the CTA
        int k_free = ntiles - KB, v_free = ntiles - VB;
        auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_bounded(b, parity, kWaitNs); };
        auto issue_s = [&](int x, bool last) {
#pragma unroll
          for (int box = 0; box < C::kBoxes; ++box)
            mma4_ss(tmem + C::kColS + C::kKv * x, dQ + ((x * C::kQBytes + box * C::kQBox) >> 4),
                    dK + ((kr.stage * C::kTile + box * C::kBox) >> 4), idS, box > 0);
          tc::commit(bar(kBarS + x));
          if (last) {
            if (k_free-- > 0) tc::commit(bar(kKFree + kr.stage));
            kr.next(KB);
          }
        };
        // O_x (+)= P_x V: 16 tokens a step, P in 8 columns each from 64 h on
        auto issue_o = [&](int x, bool first, bool last) {
#pragma unroll
          for (int h = 0; h < C::kKv / 64; ++h)
            mma4_ts(tmem + C::kColO + D * x, tmem + C::kColS + C::kKv * x + 64 * h,
                    dV + ((vr.stage * C::kTile) >> 4) + 512 * h, idO, !first || h > 0);
          tc::commit(bar(kBarO + x));
          if (last) {
            if (v_free-- > 0) tc::commit(bar(kVFree + vr.stage));
            vr.next(VB);
          }
        };
        bool ok = true;
        uint32_t par[2] = {0, 0};  // phase of each group's next product
        // Group x's products on one tile: O, and S of its next tile if there is
        // one. first_use, last_use: of the tile's V (and the next one's K).
        auto step = [&](int x, bool first, bool more, bool first_use, bool last_use) {
          // P_x (and clean V rows) written, V there; both tested before either is
          // waited for
          const bool v_in = !first_use || mbar_try_wait(bar(kVReady + vr.stage), vr.phase);
          const bool p_in = mbar_try_wait(bar(kBarP + x), par[x]);
          if (!p_in && !(ok = wait(bar(kBarP + x), par[x]))) return;
          if (!v_in && !(ok = wait(bar(kVReady + vr.stage), vr.phase))) return;
          tc::fence_after_sync();
          issue_o(x, first, last_use);
          if (more) {
            const bool k_in = !first_use || mbar_try_wait(bar(kKReady + kr.stage), kr.phase);
            if (!(ok = wait(bar(kBarO + x), par[x]))) return;  // P_x consumed
            if (!k_in && !(ok = wait(bar(kKReady + kr.stage), kr.phase))) return;
            tc::fence_after_sync();
            issue_s(x, last_use);
          }
          par[x] ^= 1;
        };
        uint32_t seg = 0;
        for (int f = f0; ok && f < f1; f += sg.nt, seg ^= 1) {
          segment_at(a, f, f1, &gi, &sg);
          if (!(ok = wait(bar(kBarQ), seg))) break;
          if (!(ok = wait(bar(kKReady + kr.stage), kr.phase))) break;
          tc::fence_after_sync();
          if (NX == 2 && sg.dual) {  // both groups on every tile
            issue_s(0, false);
            issue_s(1, true);
            for (int n = 0; ok && n < sg.nt; ++n) {
              step(0, n == 0, n + 1 < sg.nt, true, false);
              if (ok) step(1, n == 0, n + 1 < sg.nt, false, true);
            }
          } else if (NX == 2) {  // the groups on alternate tiles
            issue_s(0, true);
            if (sg.nt > 1) {
              if (!(ok = wait(bar(kKReady + kr.stage), kr.phase))) break;
              tc::fence_after_sync();
              issue_s(1, true);
            }
            for (int n = 0; ok && n < sg.nt; n += 2) {
              step(0, n == 0, n + 2 < sg.nt, true, true);
              if (ok && n + 1 < sg.nt) step(1, n == 0, n + 3 < sg.nt, true, true);
            }
          } else {
            issue_s(0, true);
            for (int n = 0; ok && n < sg.nt; ++n) step(0, n == 0, n + 1 < sg.nt, true, true);
          }
        }
        if (!ok) {
          atomicOr(a.err, PA_DEVERR_TIMEOUT);
          tc::commit(bar(kBarDrain));  // nor a product
          (void)mbar_wait_bounded(bar(kBarDrain), 0, kDrainNs);
        }
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ FP8 converters
      // e4m3 tile -> the f16 buffer: a 16-byte chunk of 16 codes becomes two
      // 16-byte chunks of f16 in the 64-dim box that holds them; V rows behind the
      // prefix become zeros. (The conversions bind a warp: about 2,000 cycles for
      // 8 KB.)
      if constexpr (FP8) {
        constexpr int kChunks = D / 16, kPer = 32 / kChunks;  // chunks a row, rows a pass
        constexpr int kOctets = C::kKv / 8;  // of rows: a warp takes every kConv-th
        const int o0 = warp - C::kConvWarp0;
        const int ch = lane % kChunks, q0 = lane / kChunks;
        const int c16 = 2 * (ch & 3);
        auto convert = [&](uint32_t src, uint32_t dst, int lim) {
          src += (ch >> 3) * C::kBox;
          dst += (ch >> 2) * C::kBox;
          // rows r, r + 8, ... share one swizzle
          static_assert(8 % kPer == 0, "passes of a row octet");
#pragma unroll 1
          for (int p = 0; p < 8 / kPer; ++p) {
            const int r0 = 8 * o0 + q0 + kPer * p;
            const uint32_t from = src + r0 * 128 + (((ch & 7) ^ (r0 & 7)) << 4);
            const uint32_t lo = dst + r0 * 128 + ((c16 ^ (r0 & 7)) << 4);
            const uint32_t hi = dst + r0 * 128 + (((c16 + 1) ^ (r0 & 7)) << 4);
#pragma unroll
            for (int k = 0; k < kOctets; k += kConv) {
              if (o0 + k >= kOctets) break;
              uint32_t w[4] = {0u, 0u, 0u, 0u}, h[8];
              if (8 * (o0 + k) < lim) lds_v4(from + 1024 * k, w[0], w[1], w[2], w[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                h[2 * i] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] & 0xffffu));
                h[2 * i + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16));
              }
              sts_v4(lo + 1024 * k, make_uint4(h[0], h[1], h[2], h[3]));
              sts_v4(hi + 1024 * k, make_uint4(h[4], h[5], h[6], h[7]));
            }
          }
        };
        bool ok = true;
        int c = 0;
        for (int f = f0; ok && f < f1; f += sg.nt) {
          segment_at(a, f, f1, &gi, &sg);
          for (int n = 0; ok && n < sg.nt; ++n, ++c) {
            const int lim = sg.g.prefix - (sg.t0 + n) * C::kKv;  // rows of the tile inside the prefix
            const uint32_t free_par = ((c - 2) >> 1) & 1;  // of the buffers' last tile
            if (!(ok = wait_all(bar(kBarKFull), c & 1))) break;
            if (c > 1 && !(ok = wait_all(bar(kBarCKFree + (c & 1)), free_par))) break;
            convert(sK, sKc + (c & 1) * C::kTile, C::kKv);
            fence_proxy_async();  // the f16 tile, visible to the tensor core
            mbar_arrive(bar(kBarCKFull + (c & 1)));
            mbar_arrive(bar(kBarKEmpty));  // reload the stage
            const uint32_t vt = sVc + (c & 1) * C::kTile;
            if (!(ok = wait_all(bar(kBarVFull), c & 1))) break;
            if (c > 1 && !(ok = wait_all(bar(kBarCVFree + (c & 1)), free_par))) break;
            convert(sV, vt, lim);
            fence_proxy_async();
            mbar_arrive(bar(kBarCVFull + (c & 1)));
            mbar_arrive(bar(kBarVEmpty));
          }
        }
        if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (C::kSplitRegs)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2;        // group
    const int r = tid - x * kRows;  // row of the tile = tensor-memory lane
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = trow + C::kColS + C::kKv * x, tO = trow + C::kColO + D * x;
    const SharedRow* rows = shared_rows(a.plan, a.ctas, a.NG);
    // Whole-warp row access: kPer rows at once, kCh lanes of 16 bytes each. A row
    // of Q (D 16-bit values) and half a row of O (D / 2 floats) have 2 D bytes.
    constexpr int kCh = D / 8, kPer = 32 / kCh;
    const int wr0 = (warp & 3) * 32;  // first row of this warp
    const int sub_r = lane / kCh, ch = lane % kCh;
    const uint32_t pair_mul = (65536u + a.G - 1) / a.G;  // row / G = row * mul >> 16, rows < 256
    bool ok = true;
    int c0 = 0, op = 0;  // products of this group so far
    uint32_t seg = 0;    // phase of the segment
    for (int f = f0; ok && f < f1; f += sg.nt, c0 += sg.nt, seg ^= 1) {
      segment_at(a, f, f1, &gi, &sg);
      const bool dual = NX == 2 && sg.dual;
      const int nj = dual || NX == 1 ? sg.nt : (sg.nt - x + 1) >> 1;  // this group's tiles
      const int u0 = dual ? x * kRows : 0;  // row of the unit (pair * G + head) at row 0 here
      float sc = fabsf(a.score_scale);
      {  // Q rows -> shared memory (K-major, 128-byte swizzle)
        const uint32_t flip = a.score_scale < 0.f ? 0x80008000u : 0u;
        const uint32_t q_tile = sQ + x * C::kQBytes + (ch >> 3) * C::kQBox;
        int sh_mine = 0;
        constexpr int kBatch = 8;  // loads in flight
#pragma unroll 1
        for (int i0 = 0; i0 < kCh; i0 += kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            // rows behind the unit's, and sequences that take no part, compute
            // on some row and are not stored
            const int ur = u0 + wr0 + (i0 + i) * kPer + sub_r;
            const int p = static_cast<int>((ur * pair_mul) >> 16), h = ur - p * a.G;
            const size_t row = static_cast<size_t>(sg.b0 + min(p, sg.np - 1)) * a.Hq +
                               static_cast<size_t>(sg.kvh) * a.G + h;
            // (no read-only load: this kernel may have started before q was written)
            v[i] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + row * D)[ch];
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int rr = wr0 + (i0 + i) * kPer + sub_r;
            if constexpr (FP8) {
              // f16 after a power-of-two rescale: largest magnitude in [2^14, 2^15)
              const uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
              float amax = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f32_of<QT>(w4[e >> 1], e & 1)));
#pragma unroll
              for (int o = kCh / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
              // 2^-sh from its exponent bits; below 2^-111 (scores that are zero
              // for any weight) the largest stays under 2^14, as does zero
              const int ex = static_cast<int>(__float_as_uint(amax) >> 23);  // 255: inf
              const int sh = ex == 255 ? 0 : max(ex - 141, -126);
              const float m = __int_as_float((127 - sh) << 23);
              const float2 m2 = make_float2(m, m);
              uint32_t o4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 t = __fmul2_rn(make_float2(f32_of<QT>(w4[e], 0), f32_of<QT>(w4[e], 1)), m2);
                o4[e] = pack16x2<false>(t.x, t.y);
              }
              v[i] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
              // to the lane that owns the row
              const int theirs = __shfl_sync(kFull, sh, (lane % kPer) * kCh);
              if (lane / kPer == i0 + i) sh_mine = theirs;
            }
            v[i].x ^= flip, v[i].y ^= flip, v[i].z ^= flip, v[i].w ^= flip;
            sts_v4(q_tile + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4), v[i]);
          }
        }
        if constexpr (FP8) sc = ldexpf(sc, sh_mine);
        fence_proxy_async();
        tc::fence_before_sync();  // the last segment's O has been read
        mbar_arrive(bar(kBarQ));
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
        // P = 2^(s * sc - ms + kLift), packed in pairs over the columns of the
        // scores just used; the last half is still in registers. It is rounded to the
        // products' 16-bit type, which the tensor core needs beside V's, against sums
        // in fp32 of the unrounded ones: at most 2^-8 of each weight for bf16 (a
        // second product for the remainders costs 15% of a 4096-token prompt's step
        // and 38% where the prefix is all), for f16 2^-11 of it and, where it is
        // subnormal, 2^-32 of the reference's weight, which the segment's largest is
        // not below. The products are added in fp32 by the tensor core, 16 tokens at
        // a time: weights below 2^-24 of a sum that is already there are lost from it
        // (55,000 tokens of weight 2^-25 behind one of weight 1: 0.1%).
        const float2 sc2 = make_float2(sc, sc), nms2 = make_float2(kLift - ms, kLift - ms);
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
          if (all_in) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 t = __ffma2_rn(score_pair(sv[i >> 4], (2 * i) & 31), sc2, nms2);
              const float p0 = ex2(t.x), p1 = ex2(t.y);
              sp[i & 3] = __fadd2_rn(sp[i & 3], make_float2(p0, p1));
              pk[i] = pack16x2<kBf16>(p0, p1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 t = __ffma2_rn(score_pair(sv[i >> 4], (2 * i) & 31), sc2, nms2);
              const bool in = 64 * hf + 2 * i < lim;
              const float p0 = in ? ex2(t.x) : 0.f, p1 = in ? ex2(t.y) : 0.f;
              sp[i & 3] = __fadd2_rn(sp[i & 3], make_float2(p0, p1));
              pk[i] = pack16x2<kBf16>(p0, p1);
            }
          }
          tc::st32(tS + 64 * hf, pk);
        }
        const float2 s01 = __fadd2_rn(sp[0], sp[1]), s23 = __fadd2_rn(sp[2], sp[3]);
        const float2 st = __fadd2_rn(s01, s23);
        l += st.x + st.y;
        if (!FP8 && !all_in && !(dual && x == 1)) {
          // the prefix ends inside this tile: zero its V rows behind it once
          // the others have landed
          const int c = c0 + n, stage = c % C::kVStages;
          if (!(ok = wait_all(bar(kBarVFull + stage), (c / C::kVStages) & 1))) break;
          const uint32_t vt = sV + stage * C::kTile;
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
      // The partials of these rows: O, its reference max and sum. They go out
      // through the Q buffer in two halves of the head dim: with its own rows, a
      // group stores both; where both groups have the same rows, each joins one
      // half of the two O (m = max(m0, m1), O = sum of 2^(mx - m) Ox, l alike)
      // and stores it.
      if (ok && nj > 0) ok = wait_all(bar(kBarO + x), (op - 1) & 1);
      const bool join = NX == 2 && !dual;
      float f_own = 1.f, f_other = 0.f;
      if (join) {
        // the same row is the same tensor-memory lane in both groups: m and l
        // change hands in columns of S, which is done with
        st2(tS, ok ? ms : kFloor, ok ? l : 0.f);
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(bar(kBarEnd));
        ok = wait_all(bar(kBarEnd), seg) && ok;
        tc::fence_after_sync();
        const float2 o = ld2(trow + C::kColS + C::kKv * (1 - x));
        const float m = fmaxf(ms, o.x);
        f_own = ex2(ms - m);
        f_other = ex2(o.x - m);
        l = l * f_own + o.y * f_other;
        ms = m;
      } else if (NX == 2) {
        mbar_arrive(bar(kBarEnd));  // keeps the phases of both kinds of segment in step
        ok = wait_all(bar(kBarEnd), seg) && ok;
      }
      tc::fence_after_sync();
      const int ur_mine = u0 + r, p_mine = static_cast<int>((ur_mine * pair_mul) >> 16);
      const bool valid = p_mine < sg.np && rows[sg.b0 + min(p_mine, sg.np - 1)].nt > 0;
      const unsigned valid_rows = __ballot_sync(kFull, valid);
      const int stride = part_stride(a.G, D);
      float* const P0 = a.part + static_cast<size_t>(sg.slot0) * stride;
      const uint64_t keep = l2_evict_last();  // the merge reads them soon
      // 16-byte chunk c of row r, where the row's own Q was: no warp touches
      // another's rows
      auto staged = [&](int row, int c) -> uint32_t {
        return sQ + x * C::kQBytes + (c >> 3) * C::kQBox + row * 128 + (((c & 7) ^ (row & 7)) << 4);
      };
      // Whether there is an O to take: uniform over the warp, and whatever it weighs
      // (a NaN in it stays one). A lone tile is group 0's.
      const bool take_own = ok && nj > 0, take_other = ok && join && (x == 1 || sg.nt > 1);
      f_own *= a.v_scale;
      f_other *= a.v_scale;
#pragma unroll 1
      for (int half = join ? x : 0; half < (join ? x + 1 : 2); ++half) {
#pragma unroll 1
        for (int d0 = 0; d0 < D / 2; d0 += 32) {
          uint32_t ov[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = 0u;
          if (take_own) {
            tc::ld32_async(tO + half * (D / 2) + d0, ov);
            tc::wait_ld(ov);
          }
          float* o = reinterpret_cast<float*>(ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f_own;
          if (take_other) {
            uint32_t ow[32];
            tc::ld32_async(trow + C::kColO + D * (1 - x) + half * (D / 2) + d0, ow);
            tc::wait_ld(ow);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fmaf(__uint_as_float(ow[i]), f_other, o[i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sts_v4(staged(r, d0 / 4 + i), make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]));
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < kCh; ++i) {
          const int lr = i * kPer + sub_r, rr = wr0 + lr;
          const int ur = u0 + rr;
          const int p = static_cast<int>((ur * pair_mul) >> 16), h = ur - p * a.G;
          uint32_t w[4];
          lds_v4(staged(rr, ch), w[0], w[1], w[2], w[3]);
          if ((valid_rows >> lr) & 1u)
            st_f32x4_hint(P0 + (p * stride + h * D + half * (D / 2) + 4 * ch),
                          make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]),
                                      __uint_as_float(w[2]), __uint_as_float(w[3])),
                          keep);
        }
        __syncwarp();
      }
      if (valid && !(join && x == 1)) {
        float* P = P0 + p_mine * stride + a.G * D + (ur_mine - p_mine * a.G);
        st_f32_hint(P, ok ? ms - kLift : kFloor, keep);
        st_f32_hint(P + a.G, ok ? l : 0.f, keep);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, PA_DEVERR_TIMEOUT);
  }

  // every MMA has completed (each group waited for its last product, or the
  // issuing thread did)
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
  if constexpr (Cfg<D, FP8>::kSplitRegs) {
    // the softmax warps wait for registers that the block must have been given
    static const int regs = [] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, prefix_attn_tc_kernel<QT, D, FP8>) == cudaSuccess ? f.numRegs : 0;
    }();
    if (2 * regs < kSoftmaxRegs + kOtherRegs) return cudaErrorLaunchOutOfResources;
  }
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
