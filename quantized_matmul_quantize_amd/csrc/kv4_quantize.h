// kv4_quantize.h -- from fp32 channels to the words of the 4-bit cache, shared
// by the calls that write it (the rule: include/qmm.h).
#pragma once

#include "kv4_device.h"

namespace qmm {

constexpr float kScaleMax16 = 65504.0f;      // largest finite binary16
// Minimum / maximum over the L consecutive lanes of a group (4, 8 or 16 lanes
// of one DPP row).
template <int L>
__device__ __forceinline__ float lanes_min(float v) {
  v = fminf(v, dpp_f<kDppXor1>(v));
  v = fminf(v, dpp_f<kDppXor2>(v));
  if constexpr (L >= 8) v = fminf(v, dpp_f<kDppHalfMirror>(v));
  if constexpr (L >= 16) v = fminf(v, dpp_f<kDppMirror>(v));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  if constexpr (L >= 8) v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  if constexpr (L >= 16) v = fmaxf(v, dpp_f<kDppMirror>(v));
  return v;
}

// Byte offset of a slot's record for head 0; false for a slot outside the cache.
__device__ __forceinline__ bool record_of(int64_t slot, const Kv4Shape& sh, uint64_t* at) {
  const int64_t id = slot >> sh.shift;
  *at = static_cast<uint64_t>(static_cast<uint32_t>(id)) *
        static_cast<uint32_t>(sh.heads * static_cast<int>(sh.record_bytes()));
  return slot >= 0 && id < sh.pages;
}

// Eight channels (one code word) of a lane; the group's range comes from its
// GROUP / 8 lanes.  The codes are those of exact division, through a correctly
// rounded reciprocal and one correction (q0 = x y, q = q0 + (x - q0 s) y is the
// correctly rounded quotient while nothing over- or underflows: s is 2^-24 ..
// 65504, and x is first held to 32 s either way, where its code is 0 or 15 all
// the same).  Rounding to an integer is the addition of 1.5 2^23.
struct CodeWord {
  uint32_t codes, param;     // binary16 scale, zero-point from bit 16
};
template <int GROUP>
__device__ __forceinline__ CodeWord quantize_word(const float (&x)[8]) {
  constexpr int kLanes = GROUP / 8;
  constexpr float kRound = 12582912.0f;                        // 1.5 2^23: the sum's low bits are the nearest integer
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  lo = lanes_min<kLanes>(lo);
  hi = lanes_max<kLanes>(hi);
  // (hi - lo) / 15, correctly rounded; beyond 2e6 the scale saturates anyway
  const float d = fminf(hi - lo, 2.0e6f);
  const float d0 = d * (1.0f / 15.0f);
  float s = fmaf(fmaf(-d0, 15.0f, d), 1.0f / 15.0f, d0);
  s = static_cast<float>(static_cast<_Float16>(fminf(s, kScaleMax16)));   // round to nearest even
  if (s == 0.0f) s = 1.0f;
  const float y = 1.0f / s, far = 32.0f * s;
  auto rounded = [&](float a) {
    a = __builtin_amdgcn_fmed3f(a, -far, far);
    const float q0 = a * y;
    return static_cast<int>(__float_as_uint(fmaf(fmaf(-q0, s, a), y, q0) + kRound));
  };
  const int bits = static_cast<int>(__builtin_bit_cast(uint32_t, kRound));
  const int z = min(max(rounded(-lo) - bits, 0), 15);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    word |= static_cast<uint32_t>(min(max(rounded(x[i]) + (z - bits), 0), 15)) << (4 * code_nibble(i));
  return {word, f32_to_f16_bits(s) | (static_cast<uint32_t>(z) << 16)};
}

// Word w of the token of a slot into its record (`head`: that of the head in
// page 0); the first lane of each group stores its param.
template <int D, int GROUP>
__device__ __forceinline__ void store_word(CodeWord c, int64_t slot, int w, bool values, const Kv4Shape& sh,
                                           uint8_t* head) {
  uint64_t at;
  if (!record_of(slot, sh, &at)) return;
  const int t = static_cast<int>(slot) & (sh.page - 1);
  uint8_t* record = head + at;
  *reinterpret_cast<uint32_t*>(record + (values ? kv4_v_word(t, w, D, sh.page) : kv4_k_word(t, w, D))) = c.codes;
  constexpr int kLanes = GROUP / 8;
  if (w % kLanes == 0)
    reinterpret_cast<uint32_t*>(record + (values ? sh.v_params() : sh.k_params()))[w / kLanes * sh.page + t] = c.param;
}

}  // namespace qmm
