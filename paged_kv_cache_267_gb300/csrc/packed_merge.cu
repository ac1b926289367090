// Join of the partial results of a ragged step's units that were cut between CTAs
// (packed_plan.cuh): with maxima m_k (log2 domain), sums l_k and unnormalised outputs
// o_k of a row's partials,
//   out = sum_k w_k o_k / sum_k w_k l_k,  w_k = 2^(m_k - max m).
// A warp takes a row: each lane reads the maxima and sums of every 32nd partial, then
// D / 32 floats of each partial, four partials in flight. The plan is read behind the
// dependency wait, as it is this step's; two dependent round trips and the partials'
// bytes through L2 bound it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_tc.cuh"
#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kFlight = 4;  // partials in flight
constexpr unsigned kFull = 0xffffffffu;

template <int OT, int D>
__global__ void __launch_bounds__(kWarps * 32) packed_merge_kernel(const PackedMergeArgs a) {
  constexpr int N = D / 32;  // floats a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  const PackedJoin j = reinterpret_cast<const PackedJoin*>(a.plan + packed_joins_at(a.ctas))[blockIdx.x];
  const size_t stride = packed_slot_floats(a.slot_rows, D);
  // rows of the unit, those of its row tiles one after the other
  for (int row = blockIdx.y * kWarps + warp; j.n > 0 && row < j.ntok * a.G; row += gridDim.y * kWarps) {
    const int tok = row / a.G, head = row - tok * a.G, xt = tok >= a.tpg ? 1 : 0;
    const int slot_row = xt * 128 + (tok - xt * a.tpg) * a.G + head;
    auto partial = [&](int k) -> const float* {
      const int slot = k == 0 ? j.slot0 : j.slot1 + 2 * (k - 1);
      return a.part + slot * stride;
    };
    float top = -INFINITY;
    for (int k = lane; k < j.n; k += 32)
      top = fmaxf(top, partial(k)[static_cast<size_t>(a.slot_rows) * D + slot_row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    float den = 0.f;
    for (int k0 = 0; k0 < j.n; k0 += 32) {
      float w = 0.f;
      if (k0 + lane < j.n) {
        const float* stat = partial(k0 + lane) + static_cast<size_t>(a.slot_rows) * D + slot_row;
        w = ex2(stat[0] - top);
        den += w * stat[a.slot_rows];
      }
      const int n = min(j.n - k0, 32);
      for (int k = 0; k < n; k += kFlight) {
        float v[kFlight][N];
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
          const float* p = partial(k0 + min(k + q, n - 1)) + static_cast<size_t>(slot_row) * D + lane * N;
          if constexpr (N == 2) {
            const float2 x = *reinterpret_cast<const float2*>(p);
            v[q][0] = x.x, v[q][1] = x.y;
          } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
              const float4 x = *reinterpret_cast<const float4*>(p + i);
              v[q][i] = x.x, v[q][i + 1] = x.y, v[q][i + 2] = x.z, v[q][i + 3] = x.w;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kFlight; ++q) {
          const float f = __shfl_sync(kFull, w, (k + q) & 31);
          if (k + q < n)
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(f, v[q][i], acc[i]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
    // an empty row is zeros; a NaN in the sum stays one
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t u[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) u[i] = pack16x2<OT == kBF16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<size_t>(j.row0 + tok) * a.out_stride +
                    static_cast<size_t>(j.kvh * a.G + head) * D + lane * N;
    if constexpr (N == 2) *reinterpret_cast<uint32_t*>(out) = u[0];
    else if constexpr (N == 4) *reinterpret_cast<uint2*>(out) = make_uint2(u[0], u[1]);
    else *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <int OT>
cudaError_t launch(const PackedMergeArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  // as many CTAs a unit as give every warp of them a row or two
  cfg.gridDim = dim3(a.ctas, a.slot_rows / (2 * kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.D == 64) return cudaLaunchKernelEx(&cfg, packed_merge_kernel<OT, 64>, a);
  if (a.D == 128) return cudaLaunchKernelEx(&cfg, packed_merge_kernel<OT, 128>, a);
  if (a.D == 256) return cudaLaunchKernelEx(&cfg, packed_merge_kernel<OT, 256>, a);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t packed_merge_launch(int out_type, const PackedMergeArgs& a, cudaStream_t s, bool pdl) {
  return out_type == kBF16 ? launch<kBF16>(a, s, pdl) : launch<kF16>(a, s, pdl);
}

}  // namespace pa
