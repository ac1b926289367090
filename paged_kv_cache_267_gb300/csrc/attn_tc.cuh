// Small device helpers of the tensor-memory attention kernels (chunk_tc.cu,
// prefix_tc.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace pa {
namespace {

__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}
// max of three (one instruction on sm_103a)
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two consecutive 32-bit tensor-memory values as an fp32 pair.
__device__ __forceinline__ float2 score_pair(const uint32_t* v, int i) {
  return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Four M128 K16 steps over one 64-element swizzled box, A and B in shared memory,
// from one asm block: step k reads both at 32 k bytes from their descriptors (in
// 16-byte units, added to the low half: the address field cannot carry). The
// first step accumulates iff acc0 != 0, the others always. (One block, so that
// the descriptors' arithmetic stays in it: with one block a step a warp spent
// about 130 cycles issuing each.)
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc0) {
  const uint32_t alo = static_cast<uint32_t>(a), ahi = static_cast<uint32_t>(a >> 32);
  const uint32_t blo = static_cast<uint32_t>(b), bhi = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n.reg .pred p0, p1;\n.reg .b32 al, bl;\n.reg .b64 ad, bd;\n"
      "setp.ne.b32 p0, %6, 0;\nsetp.eq.b32 p1, 0, 0;\n"
      "mov.b64 ad, {%1, %2};\nmov.b64 bd, {%3, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p0;\n"
      "add.u32 al, %1, 2;\nadd.u32 bl, %3, 2;\nmov.b64 ad, {al, %2};\nmov.b64 bd, {bl, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p1;\n"
      "add.u32 al, %1, 4;\nadd.u32 bl, %3, 4;\nmov.b64 ad, {al, %2};\nmov.b64 bd, {bl, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p1;\n"
      "add.u32 al, %1, 6;\nadd.u32 bl, %3, 6;\nmov.b64 ad, {al, %2};\nmov.b64 bd, {bl, %4};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p1;\n}" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc0)
      : "memory");
}
// Four M128 K16 steps with A in tensor memory: step k reads A 8 k columns on and
// B 16 k rows (2048 k bytes) on; acc0 as above.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc0) {
  const uint32_t blo = static_cast<uint32_t>(b), bhi = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n.reg .pred p0, p1;\n.reg .b32 ac, bl;\n.reg .b64 bd;\n"
      "setp.ne.b32 p0, %5, 0;\nsetp.eq.b32 p1, 0, 0;\n"
      "mov.b64 bd, {%2, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], bd, %4, p0;\n"
      "add.u32 ac, %1, 8;\nadd.u32 bl, %2, 128;\nmov.b64 bd, {bl, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %4, p1;\n"
      "add.u32 ac, %1, 16;\nadd.u32 bl, %2, 256;\nmov.b64 bd, {bl, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %4, p1;\n"
      "add.u32 ac, %1, 24;\nadd.u32 bl, %2, 384;\nmov.b64 bd, {bl, %3};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [ac], bd, %4, p1;\n}" ::"r"(d),
      "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc0)
      : "memory");
}
// 16-byte global store with an L2 cache policy.
__device__ __forceinline__ void st_f32x4_hint(float* ptr, float4 v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(ptr), "f"(v.x),
               "f"(v.y), "f"(v.z), "f"(v.w), "l"(policy)
               : "memory");
}

}  // namespace
}  // namespace pa
