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
// memory allows about ten instructions an element, so the layout keeps the
// arithmetic short: a lane holds eight elements of a head as two 8-byte chunks,
// in the rotated part four pairs (elements 4 i .. 4 i + 3 and R / 2 further on; or
// eight neighbours when interleaved), so a rotation needs no exchange between
// lanes; and a thread takes kHeads heads of the same row and kind, for which it
// folds weights and angles into four coefficients a pair once,
//   lo' = r (lo A - hi B),  hi' = r (hi C + lo E),
// A = w_lo c, B = w_hi s, C = w_hi c, E = w_lo s (behind R: c = 1, s = 0). The
// loads of all its heads are in flight together.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kManyHeads = 4;  // heads a thread in large batches
constexpr unsigned kFull = 0xffffffffu;

// Two 8-byte chunks of a head: four words of two elements.
struct Raw {
  uint32_t w[4];
};

__device__ __forceinline__ Raw load_raw(const uint16_t* head, int ea, int eb) {
  const uint2 x = *reinterpret_cast<const uint2*>(head + ea);
  const uint2 y = *reinterpret_cast<const uint2*>(head + eb);
  return Raw{{x.x, x.y, y.x, y.y}};
}
__device__ __forceinline__ void store_raw(uint16_t* head, int ea, int eb, const Raw& r) {
  *reinterpret_cast<uint2*>(head + ea) = make_uint2(r.w[0], r.w[1]);
  *reinterpret_cast<uint2*>(head + eb) = make_uint2(r.w[2], r.w[3]);
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

// Pairs of a lane's elements: pair i is (lo[i], hi[i]). Interleaved, the two of
// a word; else element i of the first chunk and of the second.
template <int ST, bool INTER>
__device__ __forceinline__ void pairs_of(const Raw& r, float2 (&lo)[2], float2 (&hi)[2]) {
  const float2 a = unpack2<ST>(r.w[0]), b = unpack2<ST>(r.w[1]);
  const float2 c = unpack2<ST>(r.w[2]), d = unpack2<ST>(r.w[3]);
  if constexpr (INTER) {
    lo[0] = make_float2(a.x, b.x), hi[0] = make_float2(a.y, b.y);
    lo[1] = make_float2(c.x, d.x), hi[1] = make_float2(c.y, d.y);
  } else {
    lo[0] = a, lo[1] = b, hi[0] = c, hi[1] = d;
  }
}

// LANES lanes a head (D <= 8 * LANES), kHeads heads of one kind a thread.
template <int ST, bool FP8, bool INTER, int LANES, int kHeads>
__global__ void __launch_bounds__(kThreads, kHeads > 1 ? 5 : 4) norm_cache_kernel(const NormCacheArgs a) {
  constexpr int kGroups = kThreads / LANES;
  // rows may come from the previous kernel, and the caches may still be read
  // by it. The next kernel may start its launch: of what is written here it
  // reads q and the caches only, behind its own wait.
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % LANES;
  const int uq = (a.Hq + kHeads - 1) / kHeads, uk = (a.Hkv + kHeads - 1) / kHeads;
  const unsigned per_row = uq + 2 * uk;
  const unsigned unit = blockIdx.x * kGroups + threadIdx.x / LANES;  // the host keeps it in 32 bits
  const unsigned row = unit / per_row;
  if (row >= static_cast<unsigned>(a.T)) return;  // whole groups: the shuffles below are per group
  const int t = static_cast<int>(row);
  const int u = static_cast<int>(unit - row * per_row);
  const int kind = u < uq ? 0 : (u < uq + uk ? 1 : 2);  // q, k, v
  const int h0 = (u - (kind == 0 ? 0 : (kind == 1 ? uq : uq + uk))) * kHeads;
  const int nh = min(kHeads, (kind == 0 ? a.Hq : a.Hkv) - h0);
  const bool on = 8 * lane < a.D, rotated = 8 * lane < a.R;
  const int ea = rotated && !INTER ? 4 * lane : 8 * lane;
  const int eb = rotated && !INTER ? (a.R >> 1) + 4 * lane : 8 * lane + 4;

  const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) +
                        t * (kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride)) +
                        h0 * a.D;
  Raw x[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    x[j] = Raw{{0u, 0u, 0u, 0u}};
    if (on && j < nh) x[j] = load_raw(src + j * a.D, ea, eb);
  }

  // where k and v go
  size_t dst = 0;  // element of head h0 in the cache
  bool stored = kind == 0;
  if (kind != 0) {
    const long long slot = a.slots[t];
    if (slot >= a.NB * a.bs) {
      if (lane == 0) atomicOr(a.err, PA_DEVERR_SLOT);
    } else if (slot >= 0) {
      stored = true;
      // pools below 2^32 slots divide in 32 bits
      const long long blk = slot >> 32 ? slot / a.bs
                                       : static_cast<unsigned>(slot) / static_cast<unsigned>(a.bs);
      dst = ((static_cast<size_t>(blk) * a.Hkv + h0) * a.bs + (slot - blk * a.bs)) * a.D;
    }
  }
  const size_t head_step = static_cast<size_t>(a.bs) * a.D;

  if (kind == 2) {
    if (!stored || !on) return;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (j >= nh) break;
      const size_t at = dst + j * head_step;
      if constexpr (FP8) {
        uint8_t* c = static_cast<uint8_t*>(a.vc) + at;
        const float2 p = unpack2<ST>(x[j].w[0]), q = unpack2<ST>(x[j].w[1]);
        const float2 r = unpack2<ST>(x[j].w[2]), s = unpack2<ST>(x[j].w[3]);
        // the IEEE quotient, as the plain write path stores it
        *reinterpret_cast<uint32_t*>(c + ea) =
            encode4(p.x / a.v_scale, p.y / a.v_scale, q.x / a.v_scale, q.y / a.v_scale);
        *reinterpret_cast<uint32_t*>(c + eb) =
            encode4(r.x / a.v_scale, r.y / a.v_scale, s.x / a.v_scale, s.y / a.v_scale);
      } else {
        store_raw(static_cast<uint16_t*>(a.vc) + at, ea, eb, x[j]);
      }
    }
    return;
  }

  // coefficients of this lane's pairs
  const void* weight = kind == 0 ? a.q_weight : a.k_weight;
  float2 A[2], B[2], C[2], E[2];
  A[0] = A[1] = C[0] = C[1] = make_float2(1.f, 1.f);  // the weights first
  if (weight && on) pairs_of<ST, INTER>(load_raw(static_cast<const uint16_t*>(weight), ea, eb), A, C);
  B[0] = B[1] = E[0] = E[1] = make_float2(0.f, 0.f);
  if (rotated) {
    int pos = a.positions[t];
    if (pos < 0 || pos >= a.NP) {
      if (lane == 0) atomicOr(a.err, PA_DEVERR_POSITION);
      pos = pos < 0 ? 0 : a.NP - 1;
    }
    const float* angle = a.cos_sin + static_cast<size_t>(pos) * a.R + 4 * lane;
    const float4 c = __ldg(reinterpret_cast<const float4*>(angle));
    const float4 s = __ldg(reinterpret_cast<const float4*>(angle + (a.R >> 1)));
    const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
    const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      B[i] = __fmul2_rn(C[i], make_float2(-s2[i].x, -s2[i].y));
      E[i] = __fmul2_rn(A[i], s2[i]);
      A[i] = __fmul2_rn(A[i], c2[i]);
      C[i] = __fmul2_rn(C[i], c2[i]);
    }
  }
  // lanes of this group within its warp
  const unsigned members = LANES == 32 ? kFull : ((1u << LANES) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
  const float inv_d = 1.f / static_cast<float>(a.D);
  const float inv_scale = kind == 1 && FP8 ? 1.f / a.k_scale : 1.f;
  // the heads' norms, interleaved: a head behind nh is zeros and goes nowhere
  float rn[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) rn[j] = 0.f;
  if (weight) {
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<ST>(x[j].w[i]);
        rn[j] = fmaf(p.x, p.x, fmaf(p.y, p.y, rn[j]));
      }
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < kHeads; ++j) rn[j] += __shfl_xor_sync(members, rn[j], o);
  }
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    float2 lo[2], hi[2];
    pairs_of<ST, INTER>(x[j], lo, hi);
    const float r = weight ? rsqrtf(fmaf(rn[j], inv_d, a.eps)) * inv_scale : inv_scale;
    const float2 r2 = make_float2(r, r);
    float2 yl[2], yh[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      yl[i] = __fmul2_rn(__ffma2_rn(hi[i], B[i], __fmul2_rn(lo[i], A[i])), r2);
      yh[i] = __fmul2_rn(__ffma2_rn(lo[i], E[i], __fmul2_rn(hi[i], C[i])), r2);
    }
    if (!on || !stored || j >= nh) continue;
    // back to element order: words of the two chunks
    const float2 w0 = INTER ? make_float2(yl[0].x, yh[0].x) : yl[0];
    const float2 w1 = INTER ? make_float2(yl[0].y, yh[0].y) : yl[1];
    const float2 w2 = INTER ? make_float2(yl[1].x, yh[1].x) : yh[0];
    const float2 w3 = INTER ? make_float2(yl[1].y, yh[1].y) : yh[1];
    if (FP8 && kind == 1) {
      uint8_t* c = static_cast<uint8_t*>(a.kc) + dst + j * head_step;
      *reinterpret_cast<uint32_t*>(c + ea) = encode4(w0.x, w0.y, w1.x, w1.y);
      *reinterpret_cast<uint32_t*>(c + eb) = encode4(w2.x, w2.y, w3.x, w3.y);
    } else {
      uint16_t* c = kind == 0 ? static_cast<uint16_t*>(a.q_out) + t * a.out_stride + (h0 + j) * a.D
                              : static_cast<uint16_t*>(a.kc) + dst + j * head_step;
      const Raw y = {{pack2<ST>(w0.x, w0.y), pack2<ST>(w1.x, w1.y), pack2<ST>(w2.x, w2.y),
                      pack2<ST>(w3.x, w3.y)}};
      store_raw(c, ea, eb, y);
    }
  }
}

template <int ST, bool FP8, bool INTER, int LANES, int kHeads>
cudaError_t launch(NormCacheArgs a, cudaStream_t s) {
  constexpr int kGroups = kThreads / LANES;
  const long long per_row = (a.Hq + kHeads - 1) / kHeads + 2ll * ((a.Hkv + kHeads - 1) / kHeads);
  // the kernel counts units in 32 bits: at most 2^31 - 2^16 a launch
  const long long most_rows = (0x7fff0000ll) / per_row;
  for (int t0 = 0, n = 0; t0 < a.T || n == 0; ++n) {
    NormCacheArgs b = a;
    b.T = static_cast<int>(a.T - t0 < most_rows ? a.T - t0 : most_rows);
    const long long grid = (b.T * per_row + kGroups - 1) / kGroups;
    b.q = static_cast<const uint16_t*>(a.q) + t0 * a.q_stride;
    b.k = static_cast<const uint16_t*>(a.k) + t0 * a.k_stride;
    b.v = static_cast<const uint16_t*>(a.v) + t0 * a.v_stride;
    b.q_out = static_cast<uint16_t*>(a.q_out) + t0 * a.out_stride;
    b.slots = a.slots + t0;
    b.positions = a.positions + t0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_cache_kernel<ST, FP8, INTER, LANES, kHeads>, b);
    if (e != cudaSuccess) return e;
    t0 += b.T;
  }
  return cudaSuccess;
}

template <int ST, bool FP8, bool INTER, int LANES>
cudaError_t launch_heads(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  // four heads a thread once that still fills every SM twice over
  const long long groups = static_cast<long long>(a.T) * (a.Hq + 2 * a.Hkv);
  const long long ctas = groups / kManyHeads / (kThreads / LANES);
  return ctas >= 2ll * num_sms ? launch<ST, FP8, INTER, LANES, kManyHeads>(a, s)
                               : launch<ST, FP8, INTER, LANES, 1>(a, s);
}

template <int ST, bool FP8, bool INTER>
cudaError_t launch_lanes(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  if (a.D <= 64) return launch_heads<ST, FP8, INTER, 8>(a, num_sms, s);
  if (a.D <= 128) return launch_heads<ST, FP8, INTER, 16>(a, num_sms, s);
  return launch_heads<ST, FP8, INTER, 32>(a, num_sms, s);
}

template <int ST>
cudaError_t launch_type(bool fp8, const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  if (a.interleaved)
    return fp8 ? launch_lanes<ST, true, true>(a, num_sms, s)
               : launch_lanes<ST, false, true>(a, num_sms, s);
  return fp8 ? launch_lanes<ST, true, false>(a, num_sms, s)
             : launch_lanes<ST, false, false>(a, num_sms, s);
}

}  // namespace

cudaError_t norm_cache_launch(int type, bool fp8, const NormCacheArgs& a, int num_sms,
                              cudaStream_t s) {
  return type == kBF16 ? launch_type<kBF16>(fp8, a, num_sms, s)
                       : launch_type<kF16>(fp8, a, num_sms, s);
}

}  // namespace pa
