// kv4.hip -- the 4-bit paged key/value cache: appending tokens, reading them
// back, copying pages.  The format and the quantization rule are stated in
// include/qmm.h; the arithmetic is that of the weight quantizer with binary16
// scales (formats.hip), for groups of channels of one token and head.

#include <algorithm>

#include "kv4_device.h"

namespace qmm {
namespace {

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

// Which (token, head, word) a thread takes: the words of a token's head on
// consecutive lanes, then four consecutive tokens (whose V words lie side by
// side), then heads; blockIdx.x the quad of tokens, blockIdx.y heads, of keys
// and then of values.  No division: they cost more than the quantization.
struct Place {
  int64_t t;
  int h, w;
  bool values;
};
template <int D>
__device__ __forceinline__ Place place_of() {
  constexpr int kWords = D / 8, kHeads = 256 / (4 * kWords);
  const int y = static_cast<int>(blockIdx.y), i = static_cast<int>(threadIdx.x);
  Place p;
  p.values = y & 1;
  p.w = i % kWords;
  p.t = static_cast<int64_t>(blockIdx.x) * 4 + i / kWords % 4;
  p.h = (y >> 1) * kHeads + i / (4 * kWords);
  return p;
}

// A thread quantizes eight channels (one code word); the group's range comes
// from its GROUP / 8 lanes.  The codes are those of exact division, through a
// correctly rounded reciprocal and one correction (q0 = x y, q = q0 + (x - q0 s) y
// is the correctly rounded quotient while nothing over- or underflows: s is
// 2^-24 .. 65504; x is held to finite numbers first, which changes no clamped
// code).  Bound by memory: 2 bytes read and 0.5 + 4 / GROUP written per channel.
template <int DT, int D, int GROUP>
__global__ __launch_bounds__(256) void kv4_append_kernel(const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs,
                                                         const uint16_t* __restrict__ v, int64_t v_ts, int64_t v_hs,
                                                         int64_t T, const int64_t* __restrict__ slots,
                                                         uint8_t* __restrict__ cache, Kv4Shape sh) {
  constexpr int kLanes = GROUP / 8;
  const Place p = place_of<D>();
  int64_t slot = -1;
  float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (p.t < T && p.h < sh.heads) {
    slot = slots[p.t];
    Vec8<DT>::load((p.values ? v + p.t * v_ts + p.h * v_hs : k + p.t * k_ts + p.h * k_hs) + 8 * p.w, x);
  }
  float lo = 0.0f, hi = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
  lo = lanes_min<kLanes>(lo);
  hi = lanes_max<kLanes>(hi);
  float s = (hi - lo) / 15.0f;
  const _Float16 s16 = static_cast<_Float16>(s >= kScaleMax16 ? kScaleMax16 : s);   // round to nearest even
  s = static_cast<float>(s16);
  if (s == 0.0f) s = 1.0f;
  const float y = 1.0f / s;
  auto quotient = [&](float a) {
    a = __builtin_amdgcn_fmed3f(a, -3.0e38f, 3.0e38f);
    const float q0 = a * y;
    return fmaf(fmaf(-q0, s, a), y, q0);
  };
  const float z = fminf(fmaxf(rintf(quotient(-lo)), 0.0f), 15.0f);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = __builtin_amdgcn_fmed3f(rintf(quotient(x[i])) + z, 0.0f, 15.0f);
    word |= static_cast<uint32_t>(c) << (4 * code_nibble(i));
  }
  const int64_t id = slot >> sh.shift;
  if (slot < 0 || id >= sh.pages) return;
  const int t = static_cast<int>(slot) & (sh.page - 1);
  uint8_t* record = cache + (id * sh.heads + p.h) * sh.record_bytes();
  *reinterpret_cast<uint32_t*>(record + (p.values ? kv4_v_word(t, p.w, D, sh.page) : kv4_k_word(t, p.w, D))) = word;
  if (p.w % kLanes == 0) {
    const uint32_t param = f32_to_f16_bits(s) | (static_cast<uint32_t>(z) << 16);
    const int g = p.w / kLanes;
    reinterpret_cast<uint32_t*>(record + (p.values ? sh.v_params() : sh.k_params()))[g * sh.page + t] = param;
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* out, int64_t i, const float x[8]) {
  if constexpr (DT == QMM_F32) {
    float* o = static_cast<float*>(out) + i;
    *reinterpret_cast<f32x4*>(o) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(o + 4) = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + i) =
        u32x4{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])};
  }
}

template <int DT, int D>
__global__ __launch_bounds__(256) void kv4_read_kernel(const uint8_t* __restrict__ cache, Kv4Shape sh,
                                                       const int64_t* __restrict__ slots, int64_t T,
                                                       void* __restrict__ k, void* __restrict__ v) {
  const Place p = place_of<D>();
  if (p.t >= T || p.h >= sh.heads) return;
  const int64_t slot = slots[p.t];
  const int64_t id = slot >> sh.shift;
  float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (slot >= 0 && id < sh.pages) {
    const int t = static_cast<int>(slot) & (sh.page - 1);
    const uint8_t* record = cache + (id * sh.heads + p.h) * sh.record_bytes();
    const uint32_t word = *reinterpret_cast<const uint32_t*>(
        record + (p.values ? kv4_v_word(t, p.w, D, sh.page) : kv4_k_word(t, p.w, D)));
    const int g = p.w >> (__builtin_ctz(sh.group) - 3);
    const uint32_t param = reinterpret_cast<const uint32_t*>(
        record + (p.values ? sh.v_params() : sh.k_params()))[g * sh.page + t];
    const float s = kv4_scale(param), z = kv4_zero(param);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (static_cast<float>(kv4_code(word, i)) - z) * s;
  }
  store8<DT>(p.values ? v : k, (p.t * sh.heads + p.h) * D + 8 * p.w, x);
}

// Page copies: blockIdx.z a layer, blockIdx.x a pair, blockIdx.y 16 KiB of
// the page, four 16-byte pieces a thread in flight.
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

// Blocks over the words of T tokens (in whole quads).
dim3 word_grid(int64_t T, const Kv4Shape& sh) {
  const int heads = 256 / (4 * (sh.D / 8));
  return dim3(static_cast<unsigned>(ceil_div(T, 4)), static_cast<unsigned>(2 * ceil_div(sh.heads, heads)));
}

template <int DT>
void launch_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, int64_t T,
                   const int64_t* slots, uint8_t* cache, const Kv4Shape& sh, hipStream_t s) {
  const uint16_t* kp = static_cast<const uint16_t*>(k);
  const uint16_t* vp = static_cast<const uint16_t*>(v);
  const dim3 grid = word_grid(T, sh);
#define QMM_APPEND(D, G) \
  kv4_append_kernel<DT, D, G><<<grid, 256, 0, s>>>(kp, k_ts, k_hs, vp, v_ts, v_hs, T, slots, cache, sh)
  switch (sh.D * 1000 + sh.group) {
    case 64032: QMM_APPEND(64, 32); break;
    case 64064: QMM_APPEND(64, 64); break;
    case 128032: QMM_APPEND(128, 32); break;
    case 128064: QMM_APPEND(128, 64); break;
    case 128128: QMM_APPEND(128, 128); break;
    case 256032: QMM_APPEND(256, 32); break;
    case 256064: QMM_APPEND(256, 64); break;
    default: QMM_APPEND(256, 128); break;
  }
#undef QMM_APPEND
}

template <int DT>
void launch_read(const uint8_t* cache, const Kv4Shape& sh, const int64_t* slots, int64_t T, void* k, void* v,
                 hipStream_t s) {
  const dim3 grid = word_grid(T, sh);
  if (sh.D == 64) kv4_read_kernel<DT, 64><<<grid, 256, 0, s>>>(cache, sh, slots, T, k, v);
  else if (sh.D == 128) kv4_read_kernel<DT, 128><<<grid, 256, 0, s>>>(cache, sh, slots, T, k, v);
  else kv4_read_kernel<DT, 256><<<grid, 256, 0, s>>>(cache, sh, slots, T, k, v);
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
  if (T >= (int64_t{1} << 31)) return QMM_ERANGE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 8) ||
      (k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7)
    return QMM_EALIGN;
  hipStream_t s = as_stream(stream);
  if (dtype == QMM_BF16)
    launch_append<QMM_BF16>(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, T, slots, cache, sh, s);
  else
    launch_append<QMM_F16>(k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, T, slots, cache, sh, s);
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
  if (T >= (int64_t{1} << 31)) return QMM_ERANGE;
  if (!aligned(cache, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 8)) return QMM_EALIGN;
  hipStream_t s = as_stream(stream);
  if (out_dtype == QMM_BF16) launch_read<QMM_BF16>(cache, sh, slots, T, k_out, v_out, s);
  else if (out_dtype == QMM_F16) launch_read<QMM_F16>(cache, sh, slots, T, k_out, v_out, s);
  else launch_read<QMM_F32>(cache, sh, slots, T, k_out, v_out, s);
  return launch_status();
}

extern "C" int kv4_copy_pages(uint8_t* cache, int64_t layers, int64_t pages, int64_t page_bytes, const int64_t* src,
                              const int64_t* dst, int64_t n, void* stream) {
  using namespace qmm;
  if (n == 0) return QMM_OK;
  if (!cache || !src || !dst || layers <= 0 || pages <= 0 || page_bytes <= 0 || n < 0) return QMM_EINVAL;
  if (!aligned(cache, 16) || page_bytes % 16 != 0 || !aligned(src, 8) || !aligned(dst, 8)) return QMM_EALIGN;
  const int64_t pieces = ceil_div(page_bytes, kCopyPieces * 256 * 16);
  if (n >= (int64_t{1} << 31) || pieces > 65535 || layers > 65535) return QMM_ERANGE;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(pieces), static_cast<unsigned>(layers));
  kv4_copy_kernel<<<grid, 256, 0, as_stream(stream)>>>(cache, pages, page_bytes, src, dst);
  return launch_status();
}
