// kv4.hip -- the 4-bit paged key/value cache: appending tokens, reading them
// back, copying pages.  The format and the quantization rule are stated in
// include/qmm.h; the arithmetic is that of the weight quantizer with binary16
// scales (formats.hip), for groups of channels of one token and head.

#include <algorithm>

#include "kv4_device.h"

namespace qmm {
namespace {

constexpr float kScaleMax16 = 65504.0f;      // largest finite binary16
// Tokens of a call: four a wavefront at the least, and a launch holds 2^24
// blocks of 256 threads.
constexpr int64_t kMostTokens = int64_t{1} << 25;

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

// How a call's words are dealt: a wavefront takes one head's words of 512 / D
// tokens at a time, NQ times; the wavefronts of a block take heads, where there
// are four, else tokens too.  blockIdx.y: heads, of keys and then of values.
// So a thread's head is uniform and its addresses are a scalar and a small
// offset: with every thread working out its own, that outweighed the rest.
struct Words {
  int heads_log2;      // wavefronts of a block over heads: 1, 2 or 4
};
struct Place {
  int64_t t0;          // first token of the wavefront
  int h, w, t;         // head, word, token within 512 / D
  bool values;
};
template <int D, int NQ>
__device__ __forceinline__ Place place_of(Words words) {
  constexpr int kWords = D / 8, kTokens = kWave / kWords;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  Place p;
  p.values = blockIdx.y & 1;
  p.w = lane % kWords;
  p.t = lane / kWords;
  p.h = static_cast<int>((blockIdx.y >> 1) << words.heads_log2) + (wave & ((1 << words.heads_log2) - 1));
  const int slice = (static_cast<int>(blockIdx.x) << (2 - words.heads_log2)) + (wave >> words.heads_log2);
  p.t0 = static_cast<int64_t>(slice) * (kTokens * NQ);
  return p;
}

// Byte offset of a slot's record for head 0; false for a slot outside the cache.
__device__ __forceinline__ bool record_of(int64_t slot, const Kv4Shape& sh, uint64_t* at) {
  const int64_t id = slot >> sh.shift;
  *at = static_cast<uint64_t>(static_cast<uint32_t>(id)) *
        static_cast<uint32_t>(sh.heads * static_cast<int>(sh.record_bytes()));
  return slot >= 0 && id < sh.pages;
}

// A thread quantizes eight channels (one code word); the group's range comes
// from its GROUP / 8 lanes.  The codes are those of exact division, through a
// correctly rounded reciprocal and one correction (q0 = x y, q = q0 + (x - q0 s) y
// is the correctly rounded quotient while nothing over- or underflows: s is
// 2^-24 .. 65504, and x is first held to 32 s either way, where its code is 0
// or 15 all the same).  Rounding to an integer is the addition of 1.5 2^23.
// Memory is 2 bytes read and 0.5 + 4 / GROUP written per channel; the ~150
// vector instructions a word take as long.  8191 tokens of 8 heads of 128 in
// groups of 64: 15.1 us, 2.9 TB/s (a large copy reaches 5.1).
template <int DT, int D, int GROUP, int NQ>
__global__ __launch_bounds__(256) void kv4_append_kernel(const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs,
                                                         const uint16_t* __restrict__ v, int64_t v_ts, int64_t v_hs,
                                                         int64_t T, const int64_t* __restrict__ slots,
                                                         uint8_t* __restrict__ cache, Kv4Shape sh, Words words) {
  constexpr int kLanes = GROUP / 8, kTokens = kWave / (D / 8);
  const Place p = place_of<D, NQ>(words);
  if (p.h >= sh.heads || p.t0 >= T) return;                    // the whole wavefront
  const uint16_t* in = p.values ? v + p.t0 * v_ts + p.h * v_hs : k + p.t0 * k_ts + p.h * k_hs;
  const int ts = static_cast<int>(p.values ? v_ts : k_ts);
  uint8_t* head = cache + p.h * sh.record_bytes();
  int64_t slot[NQ];
  float x[NQ][8];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int t = p.t + kTokens * n;
    slot[n] = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[n][i] = 0.0f;
    if (p.t0 + t < T) {
      slot[n] = slots[p.t0 + t];
      Vec8<DT>::load(in + t * ts + 8 * p.w, x[n]);
    }
  }
  constexpr float kRound = 12582912.0f;                        // 1.5 2^23: the sum's low bits are the nearest integer
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[n][i]);
      hi = fmaxf(hi, x[n][i]);
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
      word |= static_cast<uint32_t>(min(max(rounded(x[n][i]) + (z - bits), 0), 15)) << (4 * code_nibble(i));
    uint64_t at;
    if (record_of(slot[n], sh, &at)) {
      const int t = static_cast<int>(slot[n]) & (sh.page - 1);
      uint8_t* record = head + at;
      *reinterpret_cast<uint32_t*>(record + (p.values ? kv4_v_word(t, p.w, D, sh.page) : kv4_k_word(t, p.w, D))) = word;
      if (p.w % kLanes == 0) {
        const uint32_t param = f32_to_f16_bits(s) | (static_cast<uint32_t>(z) << 16);
        const int g = p.w / kLanes;
        reinterpret_cast<uint32_t*>(record + (p.values ? sh.v_params() : sh.k_params()))[g * sh.page + t] = param;
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* out, int64_t i, const float x[8]) {
  if constexpr (DT == QMM_F32) {
    float* o = static_cast<float*>(out) + i;
    *reinterpret_cast<f32x4*>(o) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i) = u32x4{
        pack_pair<DT>(x[0], x[1]), pack_pair<DT>(x[2], x[3]), pack_pair<DT>(x[4], x[5]), pack_pair<DT>(x[6], x[7])};
  }
}

// A thread expands one code word; the arithmetic is exact but for the rounding
// of the store.  Bound by memory (2 bytes written a channel) and, here, by the
// ramp of a short launch: 8191 tokens of 8 heads of 128, 11.9 us, 3.6 TB/s.
template <int DT, int D, int NQ>
__global__ __launch_bounds__(256) void kv4_read_kernel(const uint8_t* __restrict__ cache, Kv4Shape sh,
                                                       const int64_t* __restrict__ slots, int64_t T,
                                                       void* __restrict__ k, void* __restrict__ v, Words words) {
  constexpr int kTokens = kWave / (D / 8);
  const Place p = place_of<D, NQ>(words);
  if (p.h >= sh.heads || p.t0 >= T) return;                    // the whole wavefront
  const uint8_t* head = cache + p.h * sh.record_bytes();
  const int g = p.w >> (__builtin_ctz(sh.group) - 3);
  const int64_t params = (p.values ? sh.v_params() : sh.k_params()) + g * sh.page * 4;
  uint32_t word[NQ], param[NQ];
  int64_t slot[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) slot[n] = p.t0 + p.t + kTokens * n < T ? slots[p.t0 + p.t + kTokens * n] : -1;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    word[n] = param[n] = 0;                                    // scale 0: zeros for a slot outside the cache
    uint64_t at;
    if (record_of(slot[n], sh, &at)) {
      const int t = static_cast<int>(slot[n]) & (sh.page - 1);
      const uint8_t* record = head + at;
      word[n] = *reinterpret_cast<const uint32_t*>(
          record + (p.values ? kv4_v_word(t, p.w, D, sh.page) : kv4_k_word(t, p.w, D)));
      param[n] = *reinterpret_cast<const uint32_t*>(record + params + t * 4);
    }
  }
  void* out = p.values ? v : k;
  const int64_t row = (p.t0 * sh.heads + p.h) * D;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int t = p.t + kTokens * n;
    if (p.t0 + t >= T) continue;
    const float s = kv4_scale(param[n]), zs = -kv4_zero(param[n]) * s;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(static_cast<float>(kv4_code(word[n], i)), s, zs);   // (c - z) s, exactly
    store8<DT>(out, row + static_cast<int64_t>(t) * sh.heads * D + 8 * p.w, x);
  }
}

// Page copies: blockIdx.z a layer, blockIdx.x a pair, blockIdx.y 16 KiB of
// the page, four 16-byte pieces a thread in flight.  Bound by memory:
// 16 layers of 256 pages of 72 KiB, read and written, in 113 us, 5.4 TB/s.
constexpr int kCopyPieces = 4;

__global__ __launch_bounds__(256) void kv4_copy_kernel(uint8_t* __restrict__ cache, int64_t pages, int64_t page_bytes,
                                                       const int64_t* __restrict__ src,
                                                       const int64_t* __restrict__ dst) {
  const int64_t from = src[blockIdx.x], to = dst[blockIdx.x];
  if (from < 0 || from >= pages || to < 0 || to >= pages) return;
  uint8_t* layer = cache + static_cast<int64_t>(blockIdx.z) * pages * page_bytes;
  const uint8_t* a = layer + from * page_bytes;
  uint8_t* b = layer + to * page_bytes;
  const int64_t first = (static_cast<int64_t>(blockIdx.y) * kCopyPieces * 256 + threadIdx.x) * 16;
  u32x4 x[kCopyPieces];
#pragma unroll
  for (int i = 0; i < kCopyPieces; ++i) {
    const int64_t at = first + i * 256 * 16;
    if (at < page_bytes) x[i] = ld16_nt(a + at);
  }
#pragma unroll
  for (int i = 0; i < kCopyPieces; ++i) {
    const int64_t at = first + i * 256 * 16;
    if (at < page_bytes) st16_nt(b + at, x[i]);
  }
}

// Blocks over the words of T tokens, each wavefront nq times 512 / D tokens.
dim3 word_grid(int64_t T, const Kv4Shape& sh, int nq, Words* words) {
  words->heads_log2 = sh.heads >= 4 ? 2 : sh.heads >= 2 ? 1 : 0;
  const int64_t slices = ceil_div(T, 512 / sh.D * nq);
  return dim3(static_cast<unsigned>(ceil_div(slices, 4 >> words->heads_log2)),
              static_cast<unsigned>(2 * ceil_div(sh.heads, 1 << words->heads_log2)));
}
// Two words a thread from sixteen blocks a compute unit on: more bytes in
// flight, but half the blocks (8 heads of 128 in groups of 64, memory not
// cached, one and two words a thread in us: append of 2048 tokens 5.0, 5.3, of
// 4096 9.0, 8.3, of 16384 27.3, 25.8; read of 2048 4.5, 4.5, of 16384 22.7, 20.6).
bool many_tokens(int64_t T, const Kv4Shape& sh) {
  Words w;
  const dim3 g = word_grid(T, sh, 1, &w);
  return static_cast<int64_t>(g.x) * g.y >= 16 * device_cus();
}

template <int DT, int D, int GROUP>
void launch_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, int64_t T,
                   const int64_t* slots, uint8_t* cache, const Kv4Shape& sh, hipStream_t s) {
  const uint16_t* kp = static_cast<const uint16_t*>(k);
  const uint16_t* vp = static_cast<const uint16_t*>(v);
  Words w;
  if (many_tokens(T, sh)) {
    const dim3 grid = word_grid(T, sh, 2, &w);
    kv4_append_kernel<DT, D, GROUP, 2><<<grid, 256, 0, s>>>(kp, k_ts, k_hs, vp, v_ts, v_hs, T, slots, cache, sh, w);
  } else {
    const dim3 grid = word_grid(T, sh, 1, &w);
    kv4_append_kernel<DT, D, GROUP, 1><<<grid, 256, 0, s>>>(kp, k_ts, k_hs, vp, v_ts, v_hs, T, slots, cache, sh, w);
  }
}

template <int DT, typename... A>
void append_shape(const Kv4Shape& sh, A... args) {
  switch (sh.D * 1000 + sh.group) {
    case 64032: launch_append<DT, 64, 32>(args...); break;
    case 64064: launch_append<DT, 64, 64>(args...); break;
    case 128032: launch_append<DT, 128, 32>(args...); break;
    case 128064: launch_append<DT, 128, 64>(args...); break;
    case 128128: launch_append<DT, 128, 128>(args...); break;
    case 256032: launch_append<DT, 256, 32>(args...); break;
    case 256064: launch_append<DT, 256, 64>(args...); break;
    default: launch_append<DT, 256, 128>(args...); break;
  }
}

template <int DT, int D>
void launch_read(const uint8_t* cache, const Kv4Shape& sh, const int64_t* slots, int64_t T, void* k, void* v,
                 hipStream_t s) {
  Words w;
  if (many_tokens(T, sh)) {
    const dim3 grid = word_grid(T, sh, 2, &w);
    kv4_read_kernel<DT, D, 2><<<grid, 256, 0, s>>>(cache, sh, slots, T, k, v, w);
  } else {
    const dim3 grid = word_grid(T, sh, 1, &w);
    kv4_read_kernel<DT, D, 1><<<grid, 256, 0, s>>>(cache, sh, slots, T, k, v, w);
  }
}
template <int DT>
void read_shape(const uint8_t* cache, const Kv4Shape& sh, const int64_t* slots, int64_t T, void* k, void* v,
                hipStream_t s) {
  if (sh.D == 64) launch_read<DT, 64>(cache, sh, slots, T, k, v, s);
  else if (sh.D == 128) launch_read<DT, 128>(cache, sh, slots, T, k, v, s);
  else launch_read<DT, 256>(cache, sh, slots, T, k, v, s);
}

}  // namespace
}  // namespace qmm

extern "C" size_t kv4_page_bytes(int64_t kv_heads, int64_t head_dim, int64_t page, int group) {
  qmm::Kv4Shape sh;
  if (qmm::kv4_shape(1, kv_heads, head_dim, page, group, &sh) != QMM_OK) return 0;
  return static_cast<size_t>(sh.record_bytes()) * static_cast<size_t>(kv_heads);
}

extern "C" int kv4_append(const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                          int64_t v_token_stride, int64_t v_head_stride, int dtype, int64_t T, const int64_t* slots,
                          uint8_t* cache, int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page, int group,
                          void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!k || !v || !slots || !cache || T < 0 || dtype < QMM_F32 || dtype > QMM_I32) return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (dtype != QMM_BF16 && dtype != QMM_F16) return QMM_EUNSUPPORTED;
  const int64_t far = int64_t{1} << 26;          // a few tokens' distance is a 32-bit offset
  if (T >= kMostTokens || k_token_stride >= far || k_token_stride <= -far || v_token_stride >= far ||
      v_token_stride <= -far)
    return QMM_ERANGE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 8) ||
      (k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7)
    return QMM_EALIGN;
  hipStream_t s = as_stream(stream);
  if (dtype == QMM_BF16)
    append_shape<QMM_BF16>(sh, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, T, slots, cache, sh,
                           s);
  else
    append_shape<QMM_F16>(sh, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, T, slots, cache, sh,
                          s);
  return launch_status();
}

extern "C" int kv4_read(const uint8_t* cache, int64_t pages, int64_t kv_heads, int64_t head_dim, int64_t page,
                        int group, const int64_t* slots, int64_t T, void* k_out, void* v_out, int out_dtype,
                        void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!cache || !slots || !k_out || !v_out || T < 0 || out_dtype < QMM_F32 || out_dtype > QMM_I32) return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (out_dtype == QMM_I32) return QMM_EUNSUPPORTED;
  if (T >= kMostTokens) return QMM_ERANGE;
  if (!aligned(cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 8)) return QMM_EALIGN;
  hipStream_t s = as_stream(stream);
  if (out_dtype == QMM_BF16) read_shape<QMM_BF16>(cache, sh, slots, T, k_out, v_out, s);
  else if (out_dtype == QMM_F16) read_shape<QMM_F16>(cache, sh, slots, T, k_out, v_out, s);
  else read_shape<QMM_F32>(cache, sh, slots, T, k_out, v_out, s);
  return launch_status();
}

extern "C" int kv4_copy_pages(uint8_t* cache, int64_t layers, int64_t pages, int64_t page_bytes, const int64_t* src,
                              const int64_t* dst, int64_t n, void* stream) {
  using namespace qmm;
  if (n == 0) return QMM_OK;
  if (!cache || !src || !dst || layers <= 0 || pages <= 0 || page_bytes <= 0 || n < 0) return QMM_EINVAL;
  if (!aligned(cache, 16) || page_bytes % 16 != 0 || !aligned(src, 8) || !aligned(dst, 8)) return QMM_EALIGN;
  const int64_t pieces = ceil_div(page_bytes, kCopyPieces * 256 * 16);
  if (n >= (int64_t{1} << 24) || pieces > 65535 || layers > 65535) return QMM_ERANGE;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(pieces), static_cast<unsigned>(layers));
  kv4_copy_kernel<<<grid, 256, 0, as_stream(stream)>>>(cache, pages, page_bytes, src, dst);
  return launch_status();
}
