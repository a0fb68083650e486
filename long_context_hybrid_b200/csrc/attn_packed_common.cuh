// Tensor-core pieces shared by the kernels over packed prompts: packed fp32
// pairs, and 128 x 128 products of bf16 or fp16 tiles (128-byte swizzle).
#pragma once
#include "sm100.cuh"

namespace rtp {
namespace sm100 {

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > 200000000LL) return false;
  return true;
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Both operands are of the one input type: bf16, or f16 (format code 0).
template <bool F16>
__host__ __device__ constexpr uint32_t idesc(bool b_mn_major) {
  return idesc_bf16_f32(128, 128, false, b_mn_major) & (F16 ? ~((7u << 7) | (7u << 10)) : ~0u);
}
// D = A B^T of two K-major 128 x 128 tiles (8 K-steps of 16 over D = 128).
template <bool F16>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint32_t q_smem, uint32_t k_smem) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * 16384u + (kk & 3) * 32u;
    mma_bf16_ss(d_tmem, desc_sw128(q_smem + off, 16, 1024), desc_sw128(k_smem + off, 16, 1024), idesc<F16>(false),
                kk > 0 ? 1u : 0u);
  }
}
// D (+)= P V: P in TMEM (8 K-steps of 16 keys = 8 columns each), V MN-major.
template <bool F16>
__device__ __forceinline__ void issue_pv(uint32_t o_tmem, uint32_t p_tmem, uint32_t v_smem, bool accumulate) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(o_tmem, p_tmem + kk * 8u, desc_sw128(v_smem + kk * 2048u, 16384, 1024), idesc<F16>(true),
           (accumulate || kk > 0) ? 1u : 0u);
}

}  // namespace sm100
}  // namespace rtp
