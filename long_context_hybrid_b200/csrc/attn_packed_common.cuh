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
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// mbar_wait without the suspend-time hint: woken sooner (a step of the packed
// attention takes 3950 clocks with it, 4300 with the hint), and the few warps
// that wait here take few issue slots. Bounded alike.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The same for the MMA warps: on running out it only raises the flag. The
// warp then goes on through its loop (every later wait returns at once, its
// products read and write on-chip memory only, and nothing is stored), which
// keeps its control flow uniform and with it the descriptors in uniform
// registers.
// The whole warp calls it and leaves it together: a lane left behind at a
// barrier could find it a full turn further on, and wait for good.
__device__ __forceinline__ void mbar_pass(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (!mbar_test(bar, parity)) {
    const long long t0 = clock64();
    for (uint32_t it = 1; !mbar_test(bar, parity); ++it) {
      if ((it & 63u) == 0) {
        if (*abort_flag) break;
        if (clock64() - t0 > kWaitLimitCycles) {
          *abort_flag = 1;
          break;
        }
      }
    }
  }
  __syncwarp();
}

// Every thread of the cluster meets; what was written before is visible after.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of this CTA's shared-memory address in the CTA of `rank`.
__device__ __forceinline__ uint32_t remote_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void remote_st1(uint32_t addr, int x) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}
__device__ __forceinline__ void remote_st2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void remote_st4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > 200000000LL) return false;
  return true;
}
// The MMA warp runs its loop with all 32 lanes and issues under the predicate
// of one elected lane: descriptors then stay in uniform registers. Inside a
// branch of a single thread every operand takes a detour (measured: 115 clocks
// from one 128 x 128 x 16 product to the next, which itself takes 64).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(bar), "r"(on)
      : "memory");
}
// Both operands are of the one input type: bf16, or f16 (format code 0).
template <bool F16, int N = 128>
__host__ __device__ constexpr uint32_t idesc(bool b_mn_major) {
  return idesc_bf16_f32(128, N, false, b_mn_major) & (F16 ? ~((7u << 7) | (7u << 10)) : ~0u);
}
// Descriptors of 128 x 128 tiles: K-major (Q, K) and MN-major (V); a tile
// `bytes` further on is + (bytes >> 4).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t saddr) { return desc_sw128(saddr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t saddr) { return desc_sw128(saddr, 16384, 1024); }

// D = A B^T of two K-major tiles, N rows of B (8 K-steps of 16 over D = 128).
template <bool F16, int N = 128>
__device__ __forceinline__ void issue_qk(uint32_t on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint64_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
    mma_ss_if(on, d_tmem, a_desc + off, b_desc + off, idesc<F16, N>(false), kk > 0 ? 1u : 0u);
  }
}
// D (+)= P V over the 64 keys of one half of a V tile (MN-major): P in TMEM (4
// K-steps of 16 keys = 8 columns each).
template <bool F16>
__device__ __forceinline__ void issue_pv(uint32_t on, uint32_t o_tmem, uint32_t p_tmem, uint64_t v_desc, int half,
                                         bool accumulate) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int kk = half * 4 + k;
    mma_ts_if(on, o_tmem, p_tmem + k * 8u, v_desc + ((kk * 2048u) >> 4), idesc<F16>(true),
              (accumulate || k > 0) ? 1u : 0u);
  }
}

}  // namespace sm100
}  // namespace rtp
