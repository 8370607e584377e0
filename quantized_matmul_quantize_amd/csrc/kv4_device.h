// kv4_device.h -- layout of the 4-bit paged key/value cache (fixed by
// include/qmm.h), shared by its writer, its readers and the attention kernels.
//
// A record holds `page` tokens of one kv head:
//   K codes [page][D/2] | V codes [page/4][D/8][4 words] | K params [G][page] | V params [G][page]
// with G = D / group and 32-bit params (binary16 scale, zero-point from bit 16).
#pragma once

#include "qmm_device.h"

namespace qmm {

struct Kv4Shape {
  int64_t pages;
  int32_t heads, D, page, group;
  int32_t shift;   // log2(page)
  __host__ __device__ int groups() const { return D / group; }
  __host__ __device__ int64_t record_bytes() const { return static_cast<int64_t>(page) * (D + 8 * groups()); }
  __host__ __device__ int64_t k_params() const { return static_cast<int64_t>(page) * D; }
  __host__ __device__ int64_t v_params() const { return static_cast<int64_t>(page) * (D + 4 * groups()); }
};

// Status of a cache shape; fills `s` when it is supported.
inline int kv4_shape(int64_t pages, int64_t heads, int64_t D, int64_t page, int group, Kv4Shape* s) {
  if (pages <= 0 || heads <= 0 || D <= 0 || page <= 0 || group <= 0) return QMM_EINVAL;
  if (D != 64 && D != 128 && D != 256) return QMM_EUNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return QMM_EUNSUPPORTED;
  if ((group != 32 && group != 64 && group != 128) || D % group != 0) return QMM_EUNSUPPORTED;
  // page ids travel as int32, in unsigned comparisons; byte offsets are 64-bit
  if (heads > 4096 || pages >= (int64_t{1} << 31)) return QMM_ERANGE;
  *s = Kv4Shape{pages, static_cast<int32_t>(heads), static_cast<int32_t>(D), static_cast<int32_t>(page), group,
                __builtin_ctz(static_cast<unsigned>(page))};
  return QMM_OK;
}

// Byte offset in a record of code word w of the token at place t.
__device__ __forceinline__ int kv4_k_word(int t, int w, int D) {
  return t * (D / 2) + ((w & 3) * (D / 32) + (w >> 2)) * 4;
}
__device__ __forceinline__ int kv4_v_word(int t, int w, int D, int page) {
  return page * (D / 2) + (t >> 2) * (2 * D) + w * 16 + (t & 3) * 4;
}

__device__ __forceinline__ float kv4_scale(uint32_t param) { return f16lo_to_f32(param); }
__device__ __forceinline__ float kv4_zero(uint32_t param) { return static_cast<float>((param >> 16) & 0xFFu); }

// Channel e (0..7) of a code word.
__device__ __forceinline__ uint32_t kv4_code(uint32_t word, int e) { return (word >> (4 * code_nibble(e))) & 0xFu; }

}  // namespace qmm
