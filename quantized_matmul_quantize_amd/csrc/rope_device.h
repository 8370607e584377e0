// rope_device.h -- pieces of the norm and rotation of heads, shared by
// qk_norm_rope and the append with rotation.
#pragma once

#include "qmm_device.h"

namespace qmm {

// Eight consecutive channels of a 16-bit or fp32 row (the weights are read
// again by every head: ordinary loads).
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float x[8]) {
  if constexpr (DT == QMM_F32) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = a[j];
      x[j + 4] = b[j];
    }
  } else {
    const u32x4 u = ld16(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = DT == QMM_BF16 ? bf16lo_to_f32(u[j]) : f16lo_to_f32(u[j]);
      x[2 * j + 1] = DT == QMM_BF16 ? bf16hi_to_f32(u[j]) : f16hi_to_f32(u[j]);
    }
  }
}

struct HeadRows {
  const uint16_t* in;
  int64_t token_stride, head_stride;
  const void* weight;
  uint16_t* out;
  int32_t heads;
};

// Sum of the squares of a head whose channels lie eight a lane on `lanes` (a
// power of two) consecutive lanes.
__device__ __forceinline__ float head_sum_of_squares(const float x[8], int lanes) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
  if (lanes >= 2) sum += dpp_f<kDppXor1>(sum);
  if (lanes >= 4) sum += dpp_f<kDppXor2>(sum);
  if (lanes >= 8) sum += dpp_f<kDppHalfMirror>(sum);
  if (lanes >= 16) sum += dpp_f<kDppMirror>(sum);
  if (lanes >= 32) sum += __shfl_xor(sum, 16, kWave);
  if (lanes >= 64) sum += __shfl_xor(sum, 32, kWave);
  return sum;
}

// 1 / sqrt(sum / D + eps); the instruction takes subnormal numbers for 0.
__device__ __forceinline__ float inverse_rms(float sum, float inv_d, float eps) {
  const float mean = fmaf(sum, inv_d, eps);
  const bool tiny = mean < 0x1p-126f;
  return __builtin_amdgcn_rsqf(tiny ? mean * 0x1p64f : mean) * (tiny ? 0x1p32f : 1.0f);
}

}  // namespace qmm
