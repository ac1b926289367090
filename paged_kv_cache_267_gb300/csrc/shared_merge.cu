// Log-sum-exp merge of a shared-prefix decode step: the decode kernel's
// partials of every sequence's tail and the prefix kernel's of its group's
// shared positions. With maxima m_k (log2 domain), sums l_k and unnormalised
// outputs o_k of a (sequence, head)'s partials,
//   out = sum_k w_k o_k / sum_k w_k l_k,  w_k = 2^(m_k - max m).
//
// The heads of one KV head of a sequence (a pair) have the same list of
// partials, and their outputs are contiguous in each, so a CTA takes 512
// floats of a pair (four heads of 128): its warps first turn the list's maxima
// and sums into weights in shared memory, a warp a head, then each warp adds up
// its share of the partials, four of them with their sixteen loads in flight,
// and the four sums are added through shared memory. The step is bound by the
// partials' bytes through L2 and three dependent round trips (plan, maxima,
// outputs). The plain merge's half warp a column, which works out its list for
// every column, took 33 us for 8192 columns of about 8 partials.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "shared_plan.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;     // floats of a pair a CTA joins
constexpr int kList = 128;      // partials a round
constexpr int kMaxHeads = 16;   // of a pair that a chunk can meet (head_dim 64: 8)
constexpr unsigned kFull = 0xffffffffu;

template <int OT>
__global__ void __launch_bounds__(kThreads) shared_merge_kernel(const SharedMergeArgs a) {
  __shared__ float s_w[kMaxHeads][kList];
  __shared__ float s_scale[kMaxHeads];  // of what was added up before this round
  __shared__ int s_slot[kList];
  __shared__ __align__(16) float s_acc[kWarps - 1][kChunk];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int GD = a.G * a.D;
  const int chunks = (GD + kChunk - 1) / kChunk;
  const int pair = blockIdx.x / chunks, e0 = (blockIdx.x - pair * chunks) * kChunk;
  const int b = pair / a.Hkv, kvh = pair - b * a.Hkv;
  griddep_wait();  // the partials (the prefix kernel's too) are complete and visible
  if (blockIdx.x == 0 && tid == 0) {  // the decode kernel's counters, for the next step
    a.pool[0] = 0u;
    a.pool[1] = 0u;
  }
  const StepPlan pl = plan_load(a.plan);
  const int pref = a.plan[kPlanScalars + b], nt = a.plan[kPlanScalars + b + 1] - pref;
  const SharedRow row = shared_rows(a.shared, a.ctas, a.NG)[b];
  const int wsz = a.shared[kShWsz];

  const Cands cd = pair_cands(a.Hkv * pref + kvh * nt, nt, pl);
  const int tail = cd.na + cd.np;
  int n = tail, slot0 = 0, up = 0;
  if (row.nt > 0) {
    const int f0 = row.f0 + kvh * row.kv_step, w0 = f0 / wsz;
    up = row.up;
    slot0 = a.part0 + row.slot0 + (kvh * row.nut + row.lid0 + w0) * up;
    n += (f0 + row.nt - 1) / wsz - w0 + 1;
  }
  const int S = a.B * a.Hkv;
  auto slot_of = [&](int k) -> int {
    if (k < cd.na) return pair + cd.w0 + k;
    if (k < tail) return S + a.NW + pair + cd.i0 + (k - cd.na);
    return slot0 + (k - tail) * up;
  };
  const size_t stride = static_cast<size_t>(part_stride(a.G, a.D));
  const int h0 = e0 / a.D;                                        // heads of this chunk
  const int nh = min(a.G, (e0 + kChunk + a.D - 1) / a.D) - h0;

  // this lane's four groups of four floats, and their heads
  float4 acc[4];
  int head[4];
  bool on[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int e = e0 + 128 * v + 4 * lane;
    on[v] = e < GD;
    head[v] = on[v] ? e / a.D - h0 : 0;
  }
  // running maximum and sum of the heads this warp weighs (lane 0 of each)
  constexpr int kOwn = kMaxHeads / kWarps;
  float M[kOwn], den[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) M[i] = -INFINITY, den[i] = 0.f;
  const uint64_t once = l2_evict_first();  // each partial is read once

  for (int k0 = 0; k0 < n; k0 += kList) {
    const int nk = min(kList, n - k0);
    if (k0 > 0) __syncthreads();  // the last round's weights have been used
    if (tid < nk) s_slot[tid] = slot_of(k0 + tid);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int h = warp + kWarps * i;
      if (h >= nh) break;
      float m[kList / 32], l[kList / 32];
      float top = M[i];
#pragma unroll
      for (int q = 0; q < kList / 32; ++q) {
        const int k = 32 * q + lane;
        m[q] = -INFINITY;
        l[q] = 0.f;
        if (k < nk) {
          const float* P = a.part + static_cast<size_t>(slot_of(k0 + k)) * stride + GD + h0 + h;
          m[q] = ld_f32_hint(P, once);
          l[q] = ld_f32_hint(P + a.G, once);
        }
      }
#pragma unroll
      for (int q = 0; q < kList / 32; ++q) top = fmaxf(top, m[q]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kList / 32; ++q) {
        const float w = m[q] > -INFINITY ? fast_exp2(m[q] - top) : 0.f;
        s_w[h][32 * q + lane] = w;
        sum += w * l[q];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      const float old = M[i] > -INFINITY ? fast_exp2(M[i] - top) : 0.f;
      den[i] = den[i] * old + sum;
      M[i] = top;
      if (lane == 0) s_scale[h] = old;
    }
    __syncthreads();
    if (k0 > 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = s_scale[head[v]];
        acc[v].x *= f, acc[v].y *= f, acc[v].z *= f, acc[v].w *= f;
      }
    }
    // partials warp, warp + 4, ...: four in flight
    for (int k = warp; k < nk; k += 4 * kWarps) {
      float4 o[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = k + j * kWarps;
        const float* P = a.part + static_cast<size_t>(s_slot[kk < nk ? kk : k]) * stride + e0 + 4 * lane;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          o[j][v] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (kk < nk && on[v]) o[j][v] = ld_f32x4_hint(P + 128 * v, once);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = k + j * kWarps;
        if (kk >= nk) break;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float w = s_w[head[v]][kk];
          acc[v].x += w * o[j][v].x;
          acc[v].y += w * o[j][v].y;
          acc[v].z += w * o[j][v].z;
          acc[v].w += w * o[j][v].w;
        }
      }
    }
  }

  // the warps' sums, and the heads' denominators
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int h = warp + kWarps * i;
    if (h < nh && lane == 0) s_scale[h] = den[i] > 0.f ? 1.f / den[i] : 0.f;  // empty range: zeros
  }
  if (warp > 0) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<float4*>(&s_acc[warp - 1][128 * v + 4 * lane]) = acc[v];
  }
  __syncthreads();
  if (warp == 0) {
    uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<size_t>(pair) * GD + e0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float4 x = acc[v];
#pragma unroll
      for (int w = 0; w < kWarps - 1; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(&s_acc[w][128 * v + 4 * lane]);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      if (!on[v]) continue;
      const float f = s_scale[head[v]];
      uint2 u;
      if constexpr (OT == kBF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x.x * f, x.y * f);
        const __nv_bfloat162 q = __floats2bfloat162_rn(x.z * f, x.w * f);
        u = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
      } else {
        const __half2 p = __floats2half2_rn(x.x * f, x.y * f);
        const __half2 q = __floats2half2_rn(x.z * f, x.w * f);
        u = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
      }
      *reinterpret_cast<uint2*>(out + 128 * v + 4 * lane) = u;
    }
  }
}

}  // namespace

cudaError_t shared_merge_launch(int out_type, const SharedMergeArgs& a, cudaStream_t s, bool pdl) {
  const long long grid = static_cast<long long>(a.B) * a.Hkv * ((a.G * a.D + kChunk - 1) / kChunk);
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return out_type == kBF16 ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<kBF16>, a)
                           : cudaLaunchKernelEx(&cfg, shared_merge_kernel<kF16>, a);
}

}  // namespace pa
