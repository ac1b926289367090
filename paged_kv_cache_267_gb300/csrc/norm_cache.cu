// Norm of every query and key head, position rotation, and the cache write,
// in one pass over a batch's projected rows.
//
// For a head x of D elements (q with q_weight, k with k_weight):
//   y = x * w / sqrt(mean(x^2) + eps)        (y = x where there is no weight)
// and on the first R elements, pair i of R / 2 at angle row (c_i, s_i) of the
// row's position,
//   (a, b) -> (a c_i - b s_i, b c_i + a s_i)
// with (a, b) = elements (i, i + R / 2), or (2 i, 2 i + 1) when interleaved.
// q goes to q_out, k and v (v as it is) to the row's cache slot; everything
// between the load and the store is fp32 and is rounded once.
//
// The pass moves each row once in and once out. At 16 bits an element the
// memory allows about ten instructions an element, so the layout keeps them few: a
// lane holds sixteen elements of a head as two 16-byte chunks, in the rotated
// part eight pairs (elements 8 i .. 8 i + 7 and R / 2 further on; or sixteen
// neighbours when interleaved), so a rotation needs no exchange between lanes;
// and a thread takes kHeads heads of the same row and kind, for which it folds
// weights and angles into four coefficients a pair once,
//   lo' = r (lo A - hi B),  hi' = r (hi C + lo E),
// A = w_lo c, B = w_hi s, C = w_hi c, E = w_lo s (behind R: c = 1, s = 0, and the
// other element does not enter, which may be infinite). The
// loads of all its heads are in flight together; neighbouring groups of lanes
// take neighbouring heads, so that a CTA reads and writes one piece of the rows.
// 16384 rows of 32 + 2 x 8 heads of 128: 68.7 us (5.93 TB/s) into a 16-bit cache,
// 71.4 us into an e4m3 one. Half the elements a lane, 78.6 and 74 us; two heads a
// thread, 78 us; eight or more (one batch after the other), 93-130 us; a CTA
// that stays with its heads over many rows, 165 us (registers for it leave a
// quarter of the threads). No one thing bounds what is left, with 24 warps an SM and
// issue slots at 51%: 15% more instructions (no paired fp32 operations) cost 1%
// (72.3 us), a fourth CTA an SM spills (89 us), and persistent CTAs that copy the
// next unit, with its angles or without, into shared memory take 75-78 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "pa_internal.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kManyHeads = 4;  // heads a thread in large batches
constexpr unsigned kFull = 0xffffffffu;

// x / d for x < 2^31 by the host's multiplication (see FastDiv).
__device__ __forceinline__ unsigned quot31(unsigned x, const FastDiv& f) {
  return f.mul ? __umulhi(x, f.mul) >> f.shift : x;
}

// Two 16-byte chunks of a head: eight words of two elements.
struct Raw {
  uint4 a, b;
};

__device__ __forceinline__ Raw load_raw(const uint16_t* head, int ea, int eb) {
  return Raw{*reinterpret_cast<const uint4*>(head + ea), *reinterpret_cast<const uint4*>(head + eb)};
}
__device__ __forceinline__ void store_raw(uint16_t* head, int ea, int eb, const Raw& r) {
  *reinterpret_cast<uint4*>(head + ea) = r.a;
  *reinterpret_cast<uint4*>(head + eb) = r.b;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <int ST>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (ST == kBF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int ST>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (ST == kBF16) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
  } else {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
}
// e4m3 codes of four values (nearest even, saturating).
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// e4m3 codes of x / scale, the quotient as the plain write path takes it. From the
// correctly rounded reciprocal: the product q is within 1.5 ulp of the quotient, one
// fma gives its remainder (exact, or rounded in its 25th bit), and a second one
// rounds q - remainder / scale (after Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). What is rounded is off
// by less than 2^-22 ulp, so the result is the correctly rounded quotient unless
// that lies as near to the middle of two floats. The remainder is taken as q scale
// - x, and x is given negated: an exact one, +0, then leaves a zero q its sign. Holds for
// scales in [2^-60, 2^60] (what underflows is then far below the least code) and
// finite q; other scales are brought there with x by a power of two, which loses
// nothing that has a code other than zero or the largest, and x is cut to 512
// scale where any of a lane's is beyond. (The compiler's quotient made the e4m3
// write of v cost as much as the norm and rotation of q.)
struct CodeScale {
  float scale, ninv, shift;
  __device__ __forceinline__ explicit CodeScale(float s) {
    shift = s < 0x1p-60f ? 0x1p100f : (s > 0x1p60f ? 0x1p-100f : 1.f);
    scale = s * shift;
    ninv = -1.f / scale;
  }
};
__device__ __forceinline__ float clamp_nan(float x, float lim) {  // a NaN stays one
  float y;
  asm("{\n.reg .f32 t;\nmin.NaN.f32 t, %1, %2;\nmax.NaN.f32 %0, t, %3;\n}" : "=f"(y) : "f"(x), "f"(lim), "f"(-lim));
  return y;
}
// Eight codes, in order, of the negated values nx.
__device__ __forceinline__ uint2 encode8(float2 (&nx)[4], const CodeScale& s) {
  const float2 shift = make_float2(s.shift, s.shift);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    nx[i] = __fmul2_rn(nx[i], shift);
    top = fmaxf(fmaxf(fabsf(nx[i].x), fabsf(nx[i].y)), top);
  }
  if (top > 512.f * s.scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      nx[i] = make_float2(clamp_nan(nx[i].x, 512.f * s.scale), clamp_nan(nx[i].y, 512.f * s.scale));
  }
  const float2 sc = make_float2(s.scale, s.scale), ninv = make_float2(s.ninv, s.ninv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __fmul2_rn(nx[i], ninv);
    nx[i] = __ffma2_rn(__ffma2_rn(q, sc, nx[i]), ninv, q);
  }
  return make_uint2(encode4(nx[0].x, nx[0].y, nx[1].x, nx[1].y), encode4(nx[2].x, nx[2].y, nx[3].x, nx[3].y));
}

// Pairs of a lane's elements, as float2 of two pairs: pair i is (lo_i, hi_i).
// Interleaved, the two of a word; else element i of the first chunk and of the
// second. Words (2 q, 2 q + 1) of the order below make lo[q], hi[q] when
// interleaved, word q of each chunk otherwise.
template <int ST, bool INTER>
__device__ __forceinline__ void pairs_of(const Raw& r, float2 (&lo)[4], float2 (&hi)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (INTER) {
      const uint4& v = q < 2 ? r.a : r.b;
      const float2 x = unpack2<ST>(word(v, 2 * (q & 1))), y = unpack2<ST>(word(v, 2 * (q & 1) + 1));
      lo[q] = make_float2(x.x, y.x), hi[q] = make_float2(x.y, y.y);
    } else {
      lo[q] = unpack2<ST>(word(r.a, q));
      hi[q] = unpack2<ST>(word(r.b, q));
    }
  }
}
// Back to element order: the eight pairs of values of the two chunks.
template <bool INTER>
__device__ __forceinline__ void order_of(const float2 (&lo)[4], const float2 (&hi)[4], float2 (&e)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (INTER) {
      e[2 * q] = make_float2(lo[q].x, hi[q].x);
      e[2 * q + 1] = make_float2(lo[q].y, hi[q].y);
    } else {
      e[q] = lo[q];
      e[4 + q] = hi[q];
    }
  }
}

// LANES lanes a head (D <= 16 * LANES), kHeads heads of one kind a thread; PART:
// some lanes are behind R.
template <int ST, bool FP8, bool INTER, bool PART, int LANES, int kHeads>
__global__ void __launch_bounds__(kThreads, kHeads > 1 ? 3 : 4) norm_cache_kernel(const NormCacheArgs a) {
  constexpr int kGroups = kThreads / LANES;
  // rows may come from the previous kernel, and the caches may still be read
  // by it. The next kernel may start its launch: of what is written here it
  // reads q and the caches only, behind its own wait.
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % LANES;
  const int uq = (a.Hq + kHeads - 1) / kHeads, uk = (a.Hkv + kHeads - 1) / kHeads;
  const unsigned per_row = uq + 2 * uk;
  const unsigned unit = blockIdx.x * kGroups + threadIdx.x / LANES;  // the host keeps it in 31 bits
  const unsigned row = quot31(unit, a.per_row_div);
  if (row >= static_cast<unsigned>(a.T)) return;  // whole groups: the shuffles below are per group
  const int t = static_cast<int>(row);
  const int u = static_cast<int>(unit - row * per_row);
  const int kind = u < uq ? 0 : (u < uq + uk ? 1 : 2);  // q, k, v
  const int h0 = (u - (kind == 0 ? 0 : (kind == 1 ? uq : uq + uk))) * kHeads;
  const int nh = min(kHeads, (kind == 0 ? a.Hq : a.Hkv) - h0);
  const bool on = 16 * lane < a.D, rotated = 16 * lane < a.R;
  const int ea = rotated && !INTER ? 8 * lane : 16 * lane;
  const int eb = rotated && !INTER ? (a.R >> 1) + 8 * lane : 16 * lane + 8;

  const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) +
                        t * (kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride)) +
                        h0 * a.D;
  Raw x[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    x[j].a = x[j].b = make_uint4(0u, 0u, 0u, 0u);
    if (on && j < nh) x[j] = load_raw(src + j * a.D, ea, eb);
  }

  // where the results go: of head h0, and from head to head
  constexpr int elt = FP8 ? 1 : 2;
  char* dst;
  size_t step;
  bool stored = on;
  if (kind == 0) {
    dst = reinterpret_cast<char*>(static_cast<uint16_t*>(a.q_out) + t * a.out_stride + h0 * a.D);
    step = a.D * sizeof(uint16_t);
  } else {
    long long slot = a.slots[t];
    if (slot >= a.NB * a.bs) {
      if (lane == 0) atomicOr(a.err, PA_DEVERR_SLOT);
      slot = -1;
    }
    stored = stored && slot >= 0;
    if (slot < 0) slot = 0;
    const long long blk = slot >> 31 ? slot / a.bs : quot31(static_cast<unsigned>(slot), a.bs_div);
    step = static_cast<size_t>(a.bs) * a.D * elt;
    dst = static_cast<char*>(kind == 1 ? a.kc : a.vc) +
          ((static_cast<size_t>(blk) * a.Hkv + h0) * a.bs + (slot - blk * a.bs)) * (a.D * elt);
  }
  auto store_codes = [&](char* at, const float2 (&nx)[8], const CodeScale& scale) {
    float2 lo[4] = {nx[0], nx[1], nx[2], nx[3]}, hi[4] = {nx[4], nx[5], nx[6], nx[7]};
    *reinterpret_cast<uint2*>(at + ea) = encode8(lo, scale);
    *reinterpret_cast<uint2*>(at + eb) = encode8(hi, scale);
  };

  if (!FP8 && kind == 2) {  // a bit copy
    if (!stored) return;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (j >= nh) break;
      store_raw(reinterpret_cast<uint16_t*>(dst), ea, eb, x[j]);
      dst += step;
    }
    return;
  }

  // coefficients of this lane's pairs (behind R, x + -0 is x whatever its sign); v on
  // its way to codes has none
  const void* weight = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : nullptr);
  const bool turned = rotated && kind != 2;
  float2 A[4], B[4], C[4], E[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    A[q] = C[q] = make_float2(1.f, 1.f);  // the weights first
    B[q] = E[q] = make_float2(-0.f, -0.f);
  }
  if (weight && on) pairs_of<ST, INTER>(load_raw(static_cast<const uint16_t*>(weight), ea, eb), A, C);
  if (turned) {
    int pos = a.positions[t];
    if (pos < 0 || pos >= a.NP) {
      if (lane == 0) atomicOr(a.err, PA_DEVERR_POSITION);
      pos = pos < 0 ? 0 : a.NP - 1;
    }
    // (no read-only loads: this kernel may have started before they were written)
    const float4* angle = reinterpret_cast<const float4*>(a.cos_sin + static_cast<size_t>(pos) * a.R + 8 * lane);
    const float4 c0 = angle[0], c1 = angle[1], s0 = angle[a.R >> 3], s1 = angle[(a.R >> 3) + 1];
    const float2 c2[4] = {make_float2(c0.x, c0.y), make_float2(c0.z, c0.w), make_float2(c1.x, c1.y),
                          make_float2(c1.z, c1.w)};
    const float2 s2[4] = {make_float2(s0.x, s0.y), make_float2(s0.z, s0.w), make_float2(s1.x, s1.y),
                          make_float2(s1.z, s1.w)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      B[q] = __fmul2_rn(C[q], make_float2(-s2[q].x, -s2[q].y));
      E[q] = __fmul2_rn(A[q], s2[q]);
      A[q] = __fmul2_rn(A[q], c2[q]);
      C[q] = __fmul2_rn(C[q], c2[q]);
    }
  }
  // the heads' norms, interleaved: a head behind nh is zeros and goes nowhere
  const float inv_d = 1.f / static_cast<float>(a.D);
  float rn[kHeads];
  if (weight) {
    const unsigned members =
        LANES == 32 ? kFull : ((1u << LANES) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 p = unpack2<ST>(word(i < 4 ? x[j].a : x[j].b, i & 3));
        ss = __ffma2_rn(p, p, ss);
      }
      rn[j] = ss.x + ss.y;
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < kHeads; ++j) rn[j] += __shfl_xor_sync(members, rn[j], o);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) rn[j] = rsqrtf(fmaf(rn[j], inv_d, a.eps));
  } else {
#pragma unroll
    for (int j = 0; j < kHeads; ++j) rn[j] = 1.f;
  }
  // The codes apart from q's 16 bits (in one loop with a branch 74 us, not 71), but
  // those of k and v together: heads of both are in one warp, and v with codes of
  // its own beside k's took 75.
  auto finish = [&](auto is_code) {
    const CodeScale scale(!is_code.value ? 1.f : (kind == 1 ? a.k_scale : a.v_scale));
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      float2 lo[4], hi[4], yl[4], yh[4], e[8];
      pairs_of<ST, INTER>(x[j], lo, hi);
      // (codes are made of the negated values)
      const float2 r2 = is_code.value ? make_float2(-rn[j], -rn[j]) : make_float2(rn[j], rn[j]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool cross = (!PART && !is_code.value) || turned;
        const float2 h = cross ? hi[q] : make_float2(0.f, 0.f), l = cross ? lo[q] : make_float2(0.f, 0.f);
        yl[q] = __fmul2_rn(__ffma2_rn(h, B[q], __fmul2_rn(lo[q], A[q])), r2);
        yh[q] = __fmul2_rn(__ffma2_rn(l, E[q], __fmul2_rn(hi[q], C[q])), r2);
      }
      order_of<INTER>(yl, yh, e);
      if (stored && j < nh) {
        if constexpr (is_code.value) {
          store_codes(dst, e, scale);
        } else {
          Raw y;
          y.a = make_uint4(pack2<ST>(e[0].x, e[0].y), pack2<ST>(e[1].x, e[1].y), pack2<ST>(e[2].x, e[2].y),
                           pack2<ST>(e[3].x, e[3].y));
          y.b = make_uint4(pack2<ST>(e[4].x, e[4].y), pack2<ST>(e[5].x, e[5].y), pack2<ST>(e[6].x, e[6].y),
                           pack2<ST>(e[7].x, e[7].y));
          store_raw(reinterpret_cast<uint16_t*>(dst), ea, eb, y);
        }
      }
      dst += step;
    }
  };
  if constexpr (FP8) {
    if (kind > 0) {
      finish(std::true_type{});
      return;
    }
  }
  finish(std::false_type{});
}

template <int ST, bool FP8, bool INTER, bool PART, int LANES, int kHeads>
cudaError_t launch(NormCacheArgs a, cudaStream_t s) {
  constexpr int kGroups = kThreads / LANES;
  const long long per_row = (a.Hq + kHeads - 1) / kHeads + 2ll * ((a.Hkv + kHeads - 1) / kHeads);
  // the kernel counts units in 31 bits
  const long long most_rows = 0x7fff0000ll / per_row;
  for (long long t0 = 0; t0 < a.T; t0 += most_rows) {
    NormCacheArgs b = a;
    b.T = static_cast<int>(a.T - t0 < most_rows ? a.T - t0 : most_rows);
    b.q = static_cast<const uint16_t*>(a.q) + t0 * a.q_stride;
    b.k = static_cast<const uint16_t*>(a.k) + t0 * a.k_stride;
    b.v = static_cast<const uint16_t*>(a.v) + t0 * a.v_stride;
    b.q_out = static_cast<uint16_t*>(a.q_out) + t0 * a.out_stride;
    b.slots = a.slots + t0;
    b.positions = a.positions + t0;
    b.per_row_div = fast_div(static_cast<uint32_t>(per_row));
    b.bs_div = fast_div(static_cast<uint32_t>(a.bs));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((b.T * per_row + kGroups - 1) / kGroups));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_cache_kernel<ST, FP8, INTER, PART, LANES, kHeads>, b);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int ST, bool FP8, bool INTER, bool PART, int LANES>
cudaError_t launch_heads(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  // several heads a thread once that still fills every SM twice over
  const long long groups = static_cast<long long>(a.T) * (a.Hq + 2 * a.Hkv);
  const long long ctas = groups / kManyHeads / (kThreads / LANES);
  return ctas >= 2ll * num_sms ? launch<ST, FP8, INTER, PART, LANES, kManyHeads>(a, s)
                               : launch<ST, FP8, INTER, PART, LANES, 1>(a, s);
}

template <int ST, bool FP8, bool INTER, bool PART>
cudaError_t launch_lanes(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  if (a.D <= 64) return launch_heads<ST, FP8, INTER, PART, 4>(a, num_sms, s);
  if (a.D <= 128) return launch_heads<ST, FP8, INTER, PART, 8>(a, num_sms, s);
  return launch_heads<ST, FP8, INTER, PART, 16>(a, num_sms, s);
}

template <int ST, bool FP8, bool INTER>
cudaError_t launch_part(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  return a.R < a.D ? launch_lanes<ST, FP8, INTER, true>(a, num_sms, s)
                   : launch_lanes<ST, FP8, INTER, false>(a, num_sms, s);
}

template <int ST>
cudaError_t launch_type(bool fp8, const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  if (a.interleaved)
    return fp8 ? launch_part<ST, true, true>(a, num_sms, s) : launch_part<ST, false, true>(a, num_sms, s);
  return fp8 ? launch_part<ST, true, false>(a, num_sms, s) : launch_part<ST, false, false>(a, num_sms, s);
}

}  // namespace

cudaError_t norm_cache_launch(int type, bool fp8, const NormCacheArgs& a, int num_sms,
                              cudaStream_t s) {
  return type == kBF16 ? launch_type<kBF16>(fp8, a, num_sms, s)
                       : launch_type<kF16>(fp8, a, num_sms, s);
}

}  // namespace pa
