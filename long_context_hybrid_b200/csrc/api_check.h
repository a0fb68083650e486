// Host-side checks of arguments shared by the C entry points.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rtp.h"
#include "rtp_common.cuh"

namespace rtp {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline bool stride_ok(rtp_strides s) { return s.b % 8 == 0 && s.n % 8 == 0 && s.h % 8 == 0 && s.b >= 0 && s.n >= 0 && s.h >= 0; }

inline rtp_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RTP_OK : RTP_ERR_CUDA; }

// The device must be a Blackwell datacenter part (compute capability 10.x).
inline rtp_status check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return RTP_ERR_CUDA;
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return RTP_ERR_CUDA;
  return major == 10 ? RTP_OK : RTP_ERR_UNSUPPORTED;
}

inline rtp_status check_heads(const int32_t* heads, int n, int H) {
  if (!heads || n < 1 || n > kMaxHeads) return RTP_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (heads[i] < 0 || heads[i] >= H) return RTP_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    for (int k = i + 1; k < n; ++k)
      if (heads[i] == heads[k]) return RTP_ERR_INVALID_ARG;
  return RTP_OK;
}

}  // namespace rtp
