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
// The pass moves each row once in and once out and does about ten operations
// an element, so it is bound by memory: a head is held by D / 8 lanes with
// one 16-byte load each, and a thread takes kHeads heads of the same row so
// that as many loads are in flight at once and the row's angles and weights,
// which come through L1, are loaded once for all of them. The partner of a
// rotated pair is R / 16 lanes away; it is fetched as raw 16-bit data (four
// shuffles instead of eight).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"
#include "ptx.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

template <int ST>
__device__ __forceinline__ void unpack8(uint4 r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ST == kBF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
}

template <int ST>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ST == kBF16) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    } else {
      const __half2 t = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// e4m3 codes of f / scale (IEEE fp32 quotient, nearest even, saturating), as
// the plain write path stores them.
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float scale) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo)
        : "f"(f[4 * j + 1] / scale), "f"(f[4 * j] / scale));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi)
        : "f"(f[4 * j + 3] / scale), "f"(f[4 * j + 2] / scale));
    w[j] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// LANES lanes a head (D <= 8 * LANES), kHeads heads a thread.
template <int ST, bool FP8, int LANES, int kHeads>
__global__ void __launch_bounds__(kThreads) norm_cache_kernel(const NormCacheArgs a) {
  constexpr int kGroups = kThreads / LANES;
  // rows may come from the previous kernel, and the caches may still be read
  // by it. The next kernel may start its launch: of what is written here it
  // reads q and the caches only, behind its own wait.
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % LANES;
  const int heads = a.Hq + 2 * a.Hkv;
  const int per_row = (heads + kHeads - 1) / kHeads;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LANES;
  // a group behind the last unit works on the last row and stores nothing:
  // every lane of a warp takes part in the shuffles
  const bool live = unit < static_cast<long long>(a.T) * per_row;
  const int t = live ? static_cast<int>(unit / per_row) : a.T - 1;
  const int h0 = live ? static_cast<int>(unit - static_cast<long long>(t) * per_row) * kHeads : heads;
  const int e0 = 8 * lane;  // first element of this lane
  const bool on = e0 < a.D;

  uint4 raw[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = h0 + j;
    raw[j] = make_uint4(0u, 0u, 0u, 0u);
    if (!on || h >= heads) continue;
    const uint16_t* src;
    if (h < a.Hq)
      src = static_cast<const uint16_t*>(a.q) + t * a.q_stride + h * a.D;
    else if (h < a.Hq + a.Hkv)
      src = static_cast<const uint16_t*>(a.k) + t * a.k_stride + (h - a.Hq) * a.D;
    else
      src = static_cast<const uint16_t*>(a.v) + t * a.v_stride + (h - a.Hq - a.Hkv) * a.D;
    raw[j] = *reinterpret_cast<const uint4*>(src + e0);
  }

  long long slot = a.slots[t];
  if (slot >= a.NB * a.bs) {
    if (live && lane == 0 && h0 == 0) atomicOr(a.err, PA_DEVERR_SLOT);
    slot = -1;
  }
  const bool rotated = on && e0 < a.R;
  float co[8], si[8];  // of this lane's elements
  const int half = a.R >> 1;
  bool upper = false;  // this lane holds the second elements of its pairs
  if (h0 < a.Hq + a.Hkv && rotated) {
    int pos = a.positions[t];
    if (pos < 0 || pos >= a.NP) {
      if (lane == 0) atomicOr(a.err, PA_DEVERR_POSITION);
      pos = pos < 0 ? 0 : a.NP - 1;
    }
    const float* row = a.cos_sin + static_cast<size_t>(pos) * a.R;
    if (a.interleaved) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
      co[0] = co[1] = c.x, co[2] = co[3] = c.y, co[4] = co[5] = c.z, co[6] = co[7] = c.w;
      si[0] = si[1] = s.x, si[2] = si[3] = s.y, si[4] = si[5] = s.z, si[6] = si[7] = s.w;
    } else {
      upper = e0 >= half;
      const int i0 = upper ? e0 - half : e0;
      load8(row + i0, co);
      load8(row + half + i0, si);
    }
  }
  // lane (of the warp) that holds the partners
  const int hop = a.R >> 4;
  const int mate = (threadIdx.x & 31) + (!rotated || a.interleaved ? 0 : (upper ? -hop : hop));
  const int em = rotated && !a.interleaved ? (upper ? e0 - half : e0 + half) : e0;

  int kind = -1;  // whose weights w, wm hold: 0 q, 1 k
  float w[8], wm[8];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = h0 + j;
    const bool is_v = h >= a.Hq + a.Hkv;
    const bool is_q = h < a.Hq;
    float f[8];
    unpack8<ST>(raw[j], f);
    const void* weight = is_q ? a.q_weight : a.k_weight;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    uint4 other;
    other.x = __shfl_sync(kFull, raw[j].x, mate);
    other.y = __shfl_sync(kFull, raw[j].y, mate);
    other.z = __shfl_sync(kFull, raw[j].z, mate);
    other.w = __shfl_sync(kFull, raw[j].w, mate);
    if (!on || h >= heads) continue;
    if (!is_v) {
      float g[8];
      unpack8<ST>(other, g);
      if (weight) {
        if (kind != static_cast<int>(!is_q)) {
          kind = !is_q;
          unpack8<ST>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + e0)), w);
          unpack8<ST>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(weight) + em)), wm);
        }
        const float r = 1.f / sqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          f[i] = f[i] * r * w[i];
          g[i] = g[i] * r * wm[i];
        }
      }
      if (rotated) {
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float x = f[i], y = f[i + 1];
            f[i] = x * co[i] - y * si[i];
            f[i + 1] = y * co[i] + x * si[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = f[i] * co[i] + (upper ? g[i] : -g[i]) * si[i];
        }
      }
    }
    if (is_q) {
      uint16_t* dst = static_cast<uint16_t*>(a.q_out) + t * a.out_stride + h * a.D;
      *reinterpret_cast<uint4*>(dst + e0) = pack8<ST>(f);
    } else if (slot >= 0) {
      const long long blk = slot / a.bs;
      const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
      const size_t dst = ((static_cast<size_t>(blk) * a.Hkv + hk) * a.bs + (slot - blk * a.bs)) * a.D + e0;
      void* cache = is_v ? a.vc : a.kc;
      if constexpr (FP8)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst) =
            encode8(f, is_v ? a.v_scale : a.k_scale);
      else
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + dst) = is_v ? raw[j] : pack8<ST>(f);
    }
  }
}

template <int ST, bool FP8, int LANES, int kHeads>
cudaError_t launch(const NormCacheArgs& a, cudaStream_t s) {
  const int per_row = (a.Hq + 2 * a.Hkv + kHeads - 1) / kHeads;
  const long long groups = static_cast<long long>(a.T) * per_row;
  const long long grid = (groups + kThreads / LANES - 1) / (kThreads / LANES);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_cache_kernel<ST, FP8, LANES, kHeads>, a);
}

template <int ST, bool FP8, int LANES>
cudaError_t launch_heads(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  // four heads a thread once that still fills every SM twice over
  const long long groups = static_cast<long long>(a.T) * (a.Hq + 2 * a.Hkv);
  const long long ctas4 = groups / 4 / (kThreads / LANES);
  return ctas4 >= 2ll * num_sms ? launch<ST, FP8, LANES, 4>(a, s) : launch<ST, FP8, LANES, 1>(a, s);
}

template <int ST, bool FP8>
cudaError_t launch_lanes(const NormCacheArgs& a, int num_sms, cudaStream_t s) {
  if (a.D <= 64) return launch_heads<ST, FP8, 8>(a, num_sms, s);
  if (a.D <= 128) return launch_heads<ST, FP8, 16>(a, num_sms, s);
  return launch_heads<ST, FP8, 32>(a, num_sms, s);
}

}  // namespace

cudaError_t norm_cache_launch(int type, bool fp8, const NormCacheArgs& a, int num_sms,
                              cudaStream_t s) {
  if (type == kBF16)
    return fp8 ? launch_lanes<kBF16, true>(a, num_sms, s) : launch_lanes<kBF16, false>(a, num_sms, s);
  return fp8 ? launch_lanes<kF16, true>(a, num_sms, s) : launch_lanes<kF16, false>(a, num_sms, s);
}

}  // namespace pa
