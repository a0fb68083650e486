// Device view of a paged key-value cache and of packed sequences, shared by
// the serving kernels (packed prompts, paged cache).
//
// Slot s of sequence b lives in page table[b][s / page_size] at row
// s % page_size. Page ids outside [0, num_pages) are never followed: their
// slots hold no token for the kernels that read, and are not written.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rtp_common.cuh"
#include "rtp_internal.h"

namespace rtp {

// Length of sequence b, within what the call and the table can hold.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int max_len) {
  const int n = __ldg(lens + b);
  return n < 0 ? 0 : (n < max_len ? n : max_len);
}

// Page of slot s of sequence b, or -1.
__device__ __forceinline__ int page_of(const PagedView& c, int b, int64_t s) {
  const int id = __ldg(c.table + (int64_t)b * c.table_stride + (s >> c.page_shift));
  return (unsigned)id < (unsigned)c.num_pages ? id : -1;
}

// Last i in [0, n) with f(i) <= t, or -1 (f non-decreasing). The whole warp
// calls it with one t: 32 entries are probed at a time, so the loads of a step
// are independent (one round trip for 32 entries, two for 1024).
template <class F>
__device__ __forceinline__ int warp_last_le(F f, int n, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < n && f(lo + at) <= t));
    if (k == 0) return -1;
    const int skip = (k - 1) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo + __popc(__ballot_sync(0xffffffffu, lane < n && f(lo + lane) <= t)) - 1;
}

// Tiles of kRows (a power of two) rows of packed sequences without a list:
// sequence i owns the tile numbers floor(cu[i] / kRows) + i .. floor(cu[i+1] /
// kRows) + i, which are at least ceil(len / kRows) of them, so floor(T / kRows) +
// S numbers cover any lengths. Finds a number's sequence [c0, c0 + n) (row
// numbers clamped to [0, T]) and its first row within the sequence; false where
// there is none.
template <int kRows>
__device__ __forceinline__ bool packed_tile(const int32_t* cu, int S, int T, int64_t number, int* c0, int* n,
                                            int* row0) {
  static_assert((kRows & (kRows - 1)) == 0, "tiles start at multiples");
  constexpr int kShift = kRows == 128 ? 7 : 8;
  static_assert(1 << kShift == kRows, "128 or 256 rows");
  auto at = [&](int x) -> int { return min(max(__ldg(cu + x), 0), T); };
  const int i = warp_last_le([&](int x) -> int64_t { return (int64_t)(at(x) >> kShift) + x; }, S, number);
  if (i < 0) return false;
  const int a = at(i), b = at(i + 1);
  *c0 = a;
  *n = b > a ? b - a : 0;
  const int64_t r = (number - ((a >> kShift) + (int64_t)i)) << kShift;
  *row0 = (int)r;
  return r >= 0 && r < *n;                     // offsets that decrease end up on either side
}

// 16-bit element types of the serving kernels.
template <bool F16>
struct Elem16 {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
  static __device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
template <>
struct Elem16<true> {
  using T = __half;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
};

}  // namespace rtp
