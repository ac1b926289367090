// Log-sum-exp merge of a shared-prefix decode step: the decode kernel's
// partials of every sequence's tail and the prefix kernel's of its group's
// shared positions. With maxima m_k (log2 domain), sums l_k and unnormalised
// outputs o_k of a (sequence, head)'s partials,
//   out = sum_k w_k o_k / sum_k w_k l_k,  w_k = 2^(m_k - max m).
//
// The heads of one KV head of a sequence (a pair) have the same list of
// partials, and their outputs are contiguous in each, so a warp takes 512 floats
// of a pair (four heads of 128), sixteen a lane: it works out the list once,
// reads the maxima and sums of 32 partials a lane each, and adds up the
// outputs, four partials (sixteen 16-byte loads a lane) in flight, the first
// four of them while the maxima are still on their way. Two dependent round
// trips (plan, partials) and the partials' bytes through L2 bound it. Steps with
// few pairs give each task four warps, which share its list and are joined
// through shared memory. The list is worked out before the dependency wait, from
// the plan, which is complete by then. From the end of the wait: 3.3 us for 512 pairs
// of about 7 partials, 4.2 us for 2048 pairs of about 5. (A half warp a column,
// which works out the list for every column, took 33 us for 8192 columns of about
// 8 partials; a CTA a pair with the weights in shared memory first, 17 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pa_internal.h"
#include "ptx.cuh"
#include "shared_plan.cuh"
#include "step_ops.h"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 512;   // floats of a pair a task joins
constexpr int kFlight = 4;    // partials in flight
constexpr unsigned kFull = 0xffffffffu;

template <int OT, int D, int WPT>
__global__ void __launch_bounds__(kThreads, 4) shared_merge_kernel(const SharedMergeArgs a) {
  constexpr int NH = kChunk / D;  // heads a chunk
  constexpr int C = 32 / NH;      // lanes a head, where maxima and sums are read
  constexpr int kLog2D = D == 64 ? 6 : (D == 128 ? 7 : 8);
  __shared__ __align__(16) float s_acc[WPT > 1 ? kWarps - 1 : 1][kChunk];
  __shared__ float s_m[kWarps][NH], s_l[kWarps][NH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int GD = a.G * D;
  const int chunks = (GD + kChunk - 1) / kChunk;
  int task = WPT > 1 ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * kWarps + warp;
  const bool idle = task >= a.B * a.Hkv * chunks;  // whole warps, and WPT == 1
  if (idle) task = 0;
  const int pair = chunks == 1 ? task : task / chunks, e0 = (task - pair * chunks) * kChunk;
  const int b = pair / a.Hkv, kvh = pair - b * a.Hkv;
  // Before the dependency wait: the plan is complete (the decode kernel started
  // after it).
  const SharedRow row = shared_rows(a.plan, a.ctas, a.NG)[b];
  const int wsz = a.plan[kShWsz], tail_ws = a.plan[kShTailsWs];

  // the decode kernel's partials: of the warps whose units meet the pair's tiles
  int tail = 0, tail0 = 0;
  if (row.tiles > 0) {
    const int f0 = a.Hkv * row.pref + kvh * (row.tiles + 1) + 1, w0 = f0 / tail_ws;
    tail0 = pair + w0;
    tail = (f0 + row.tiles - 1) / tail_ws - w0 + 1;
  }
  int n = tail, slot0 = 0;
  if (row.nt > 0) {
    const int f0 = row.f0 + kvh * row.kv_step, w0 = f0 / wsz;
    slot0 = a.part0 + row.slot0 + (kvh * row.nut + row.lid0 + w0) * row.up;
    n += (f0 + row.nt - 1) / wsz - w0 + 1;
  }
  const size_t stride = static_cast<size_t>(part_stride(a.G, D));
  auto partial = [&](int k) -> const float* {
    const int slot = k < tail ? tail0 + k : slot0 + (k - tail) * row.up;
    return a.part + static_cast<size_t>(slot) * stride;
  };
  const int h0 = e0 >> kLog2D;  // heads of this chunk
  const int nh = min(a.G - h0, NH);
  const int k_lo = WPT > 1 ? n * warp / WPT : 0, k_hi = WPT > 1 ? n * (warp + 1) / WPT : n;

  // this lane's four groups of four floats
  float4 acc[4];
  bool on[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    on[v] = e0 + 128 * v + 4 * lane < GD && !idle;
  }
  // value x of this lane's head in group v, from the lanes that hold x by head
  auto of_head = [&](float x, int v) -> float {
    return __shfl_sync(kFull, x, ((128 * v + 4 * lane) >> kLog2D) * C);
  };
  const int hl = lane / C, cl = lane % C;  // head and partial this lane reads
  float M = -INFINITY, den = 0.f;          // running maximum and sum of head hl
  const uint64_t once = l2_evict_first();  // each partial is read once
  // the list is worked out: this CTA has read all that it wants of the plan
  __syncthreads_or((n | slot0 | tail0) < 0);
  griddep_wait();  // the partials (the prefix kernel's too) are complete and visible
  // The next kernel may start: what it writes before it waits for this one, a
  // plan, is not read here any more. (Steps one after the other then plan during
  // the merge.)
  griddep_launch_dependents();

  for (int k0 = k_lo; k0 < k_hi; k0 += 32) {
    const int k1 = min(k0 + 32, k_hi);
    float m[NH], w[NH];  // of partials cl, cl + C, ...
#pragma unroll
    for (int q = 0; q < NH; ++q) {
      const int k = k0 + cl + C * q;
      m[q] = -INFINITY;
      w[q] = 0.f;
      if (k < k1 && hl < nh) {
        const float* P = partial(k) + GD + h0 + hl;
        m[q] = ld_f32_hint(P, once);
        w[q] = ld_f32_hint(P + a.G, once);
      }
    }
    float4 o[kFlight][4];
    auto fetch = [&](int k) {
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const bool in = k + j < k1;
        const float* P = partial(in ? k + j : k0) + e0 + 4 * lane;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          o[j][v] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (in && on[v]) o[j][v] = ld_f32x4_hint(P + 128 * v, once);
        }
      }
    };
    fetch(k0);  // while the maxima are on their way
    float top = M;
#pragma unroll
    for (int q = 0; q < NH; ++q) top = fmaxf(top, m[q]);
#pragma unroll
    for (int s = C / 2; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, s));
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < NH; ++q) {
      const float e = m[q] > -INFINITY ? fast_exp2(m[q] - top) : 0.f;
      sum += e * w[q];
      w[q] = e;
    }
#pragma unroll
    for (int s = C / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
    const float scale = M > -INFINITY ? fast_exp2(M - top) : 0.f;  // of what was added up before
    den = den * scale + sum;
    M = top;
    if (k0 > k_lo) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float f = of_head(scale, v);
        acc[v].x *= f, acc[v].y *= f, acc[v].z *= f, acc[v].w *= f;
      }
    }
#pragma unroll
    for (int i = 0; i < 32; i += kFlight) {  // partials k0 + i ..., weights in w[i / C]
      if (k0 + i >= k1) break;
      if (i > 0) fetch(k0 + i);
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const float wq = w[(i + j) / C];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          // (0 behind the list: its lane has none)
          const float f = __shfl_sync(kFull, wq, ((128 * v + 4 * lane) >> kLog2D) * C + (i + j) % C);
          acc[v].x += f * o[j][v].x;
          acc[v].y += f * o[j][v].y;
          acc[v].z += f * o[j][v].z;
          acc[v].w += f * o[j][v].w;
        }
      }
    }
  }

  if constexpr (WPT > 1) {
    if (cl == 0) s_m[warp][hl] = M, s_l[warp][hl] = den;
    if (warp > 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<float4*>(&s_acc[warp - 1][128 * v + 4 * lane]) = acc[v];
    }
    __syncthreads();
    if (warp > 0) return;
    float top = s_m[0][hl], f[kWarps];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) top = fmaxf(top, s_m[q][hl]);
    den = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      f[q] = s_m[q][hl] > -INFINITY ? fast_exp2(s_m[q][hl] - top) : 0.f;
      den += f[q] * s_l[q][hl];
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < kWarps; ++q) {
        const float4 y = q == 0 ? acc[v] : *reinterpret_cast<const float4*>(&s_acc[q - 1][128 * v + 4 * lane]);
        const float g = of_head(f[q], v);
        x.x += g * y.x, x.y += g * y.y, x.z += g * y.z, x.w += g * y.w;
      }
      acc[v] = x;
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;  // empty range: zeros
  uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<size_t>(pair) * GD + e0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float f = of_head(inv, v);
    if (!on[v]) continue;
    const float4 x = acc[v];
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

template <int OT, int D>
cudaError_t launch(const SharedMergeArgs& a, int num_sms, cudaStream_t s, bool pdl) {
  const long long tasks = static_cast<long long>(a.B) * a.Hkv * ((a.G * D + kChunk - 1) / kChunk);
  if (tasks <= 0) return cudaSuccess;
  // one warp a task once that gives every SM five of them
  const bool single = tasks >= 5ll * num_sms;
  const long long grid = single ? (tasks + kWarps - 1) / kWarps : tasks;
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
  return single ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<OT, D, 1>, a)
                : cudaLaunchKernelEx(&cfg, shared_merge_kernel<OT, D, kWarps>, a);
}

template <int OT>
cudaError_t launch_dim(const SharedMergeArgs& a, int num_sms, cudaStream_t s, bool pdl) {
  if (a.D == 64) return launch<OT, 64>(a, num_sms, s, pdl);
  if (a.D == 128) return launch<OT, 128>(a, num_sms, s, pdl);
  if (a.D == 256) return launch<OT, 256>(a, num_sms, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t shared_merge_launch(int out_type, const SharedMergeArgs& a, cudaStream_t s, bool pdl) {
  return out_type == kBF16 ? launch_dim<kBF16>(a, a.ctas, s, pdl) : launch_dim<kF16>(a, a.ctas, s, pdl);
}

}  // namespace pa
