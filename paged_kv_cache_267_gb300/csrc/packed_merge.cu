// Join of the partial results of a ragged step's units that were cut between CTAs
// (packed_plan.cuh): with maxima m_k (log2 domain), sums l_k and unnormalised outputs
// o_k of a row's partials,
//   out = sum_k w_k o_k / sum_k w_k l_k,  w_k = 2^(m_k - max m).
// A warp takes four rows, eight lanes each, so that a few partials already give every
// lane eight 16-byte loads in flight. Which unit is to be joined is in the plan, which is
// complete when this kernel starts (in small steps, whose CTAs write it, when they are
// done); CTAs without one leave at once. Two dependent round
// trips and the partials' bytes through L2 bound it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_tc.cuh"
#include "packed_ops.h"
#include "pa_internal.h"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kLanes = 8;          // a row
constexpr int kRowsWarp = 32 / kLanes;
constexpr unsigned kFull = 0xffffffffu;

template <int OT, int D>
__global__ void __launch_bounds__(kWarps * 32) packed_merge_kernel(const PackedMergeArgs a) {
  constexpr int N = D / (4 * kLanes);          // groups of four floats a lane
  constexpr int kFlight = N >= 8 ? 1 : 8 / N;  // partials in flight
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes;
  if (a.small) griddep_wait();
  const PackedJoin j = reinterpret_cast<const PackedJoin*>(a.plan + packed_joins_at(a.ctas))[blockIdx.x];
  const int row = (blockIdx.y * kWarps + warp) * kRowsWarp + lane / kLanes;
  // (one CTA stays in any case: the next kernel must not overtake the attention)
  if ((j.n == 0 || blockIdx.y * kWarps * kRowsWarp >= j.ntok * a.G) && (blockIdx.x | blockIdx.y) != 0) return;
  if (!a.small) griddep_wait();
  if (j.n == 0) return;
  // rows of the unit, those of its row tiles one after the other; lanes of rows behind
  // them work on the last one and store nothing
  const int rows = j.ntok * a.G, mine = min(row, rows - 1);
  const int tok = mine / a.G, head = mine - tok * a.G, xt = tok >= a.tpg ? 1 : 0;
  const int slot_row = xt * 128 + (tok - xt * a.tpg) * a.G + head;
  const size_t stride = packed_slot_floats(a.slot_rows, D);
  auto partial = [&](int k) -> const float* {
    return a.part + (2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * stride;
  };
  const size_t stat0 = static_cast<size_t>(a.slot_rows) * D + slot_row;
  float top = -INFINITY;
  for (int k = sub; k < j.n; k += kLanes) top = fmaxf(top, partial(k)[stat0]);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float4 acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int k0 = 0; k0 < j.n; k0 += kFlight) {
    float4 v[kFlight][N];
    float m[kFlight], l[kFlight];
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      const float* p = partial(min(k0 + q, j.n - 1));
      m[q] = k0 + q < j.n ? p[stat0] : -INFINITY;
      l[q] = p[stat0 + a.slot_rows];
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[q][i] = reinterpret_cast<const float4*>(p + static_cast<size_t>(slot_row) * D)[sub + kLanes * i];
    }
#pragma unroll
    for (int q = 0; q < kFlight; ++q) {
      if (k0 + q >= j.n) break;
      const float w = ex2(m[q] - top);
      den = fmaf(w, l[q], den);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        acc[i].x = fmaf(w, v[q][i].x, acc[i].x);
        acc[i].y = fmaf(w, v[q][i].y, acc[i].y);
        acc[i].z = fmaf(w, v[q][i].z, acc[i].z);
        acc[i].w = fmaf(w, v[q][i].w, acc[i].w);
      }
    }
  }
  if (row >= rows) return;
  // an empty row is zeros; a NaN in the sum stays one
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<size_t>(j.row0 + tok) * a.out_stride +
                  static_cast<size_t>(j.kvh * a.G + head) * D;
#pragma unroll
  for (int i = 0; i < N; ++i)
    reinterpret_cast<uint2*>(out)[sub + kLanes * i] =
        make_uint2(pack16x2<OT == kBF16>(acc[i].x * inv, acc[i].y * inv),
                   pack16x2<OT == kBF16>(acc[i].z * inv, acc[i].w * inv));
}

template <int OT>
cudaError_t launch(const PackedMergeArgs& a, cudaStream_t s, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas, a.slot_rows / (kRowsWarp * kWarps));
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
