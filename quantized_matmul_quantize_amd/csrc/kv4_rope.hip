// kv4_rope.hip -- a step's heads between the projection and the attention in
// one pass: queries normed and rotated, keys normed, rotated and appended to
// the 4-bit cache, values appended (format and rules: include/qmm.h).

#include <algorithm>

#include "kv4_quantize.h"
#include "rope_device.h"

namespace qmm {
namespace {

constexpr int kInFlight = 4;     // heads whose loads a wavefront has on their way

struct RopeAppend {
  HeadRows q, k, v;              // of v only in, strides and heads are used; q.heads may be 0
  int w_f32;                     // weights are fp32, else of the heads' type
  const int64_t* positions;
  const float* table;
  int64_t table_rows;
  int rot;
  float eps;
  const int64_t* slots;
  uint8_t* cache;
  Kv4Shape sh;
  int64_t T;
  int per;                       // heads a wavefront takes
  int q_parts, kv_parts;         // wavefronts over the heads of q, and of k (and v)
};

template <int DT>
__device__ __forceinline__ void unpack8(u32x4 u, float (&x)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = DT == QMM_BF16 ? bf16lo_to_f32(u[j]) : f16lo_to_f32(u[j]);
    x[2 * j + 1] = DT == QMM_BF16 ? bf16hi_to_f32(u[j]) : f16hi_to_f32(u[j]);
  }
}
template <int DT>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int c, float (&x)[8]) {
  if (f32) load8<QMM_F32>(w, c, x);
  else load8<DT>(w, c, x);
}

// 1 / sqrt(x) to a few units of the last place: the instruction's 24 bits and
// two Newton steps.  Zeros and infinities (and NaN) keep the instruction's result.
__device__ __forceinline__ double inverse_sqrt(double x) {
  const double r0 = __builtin_amdgcn_rsq(x);
  double r = r0;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(0.5 * r, fma(-x * r, r, 1.0), r);
  return x > 0.0 && x < __builtin_inf() ? r : r0;
}

// The wavefronts of a block share tokens (blockIdx.x: 512 / D of them, a head's
// D channels eight a lane) and take `per` heads each of one kind: cosines,
// sines and weights are read once for those.
//   Queries are in fp32, with the operations of qk_norm_rope.  Keys go from the
// input to the rounding to fp32 before the cache's rule in fp64 (a vector
// operation of gfx950 in fp64 costs what one in fp32 does): a code depends on
// which side of a border the key falls, and in fp64 that no longer depends on
// the order of the sums.  The partner's channels of a rotation by halves come as
// the 16-bit inputs and are normed again: half the exchange of fp64 values.
//   8191 tokens of 32/8 heads of 128 42 us, 181 MB at 4.3 TB/s (a copy reaches
// 5.2).  64 tokens 4.6 us: launch, the loads of slots, positions and their rows of
// the table one after another, and the norm's chain of sums.
template <int DT, int D, int GROUP, bool INTERLEAVED>
__global__ __launch_bounds__(256) void kv4_rope_append_kernel(RopeAppend a) {
  constexpr int kLanes = D / 8, kTokens = kWave / kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = threadIdx.x & (kWave - 1);
  int part = static_cast<int>(blockIdx.y) * 4 + wave;
  if (part >= a.q_parts + 2 * a.kv_parts) return;              // the whole wavefront
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + lane / kLanes;
  const bool live = t < a.T;
  const int w = lane % kLanes, c = 8 * w;                      // word of the head, first channel
  int kind = 0;                                                // q, k or v
  if (part >= a.q_parts) {
    part -= a.q_parts;
    kind = part < a.kv_parts ? 1 : 2;
    part -= kind == 1 ? 0 : a.kv_parts;
  }
  const HeadRows& rows = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
  const int first = part * a.per, end = min(first + a.per, rows.heads);
  const uint16_t* in = rows.in + (live ? t : 0) * rows.token_stride + c;
  const int64_t slot = live && kind > 0 ? a.slots[t] : -1;

  u32x4 raw[kInFlight];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int n = 0; n < kInFlight; ++n) {
      raw[n] = u32x4{0u, 0u, 0u, 0u};
      if (live && h0 + n < end) raw[n] = ld16_nt(in + (h0 + n) * rows.head_stride);
    }
  };
  if (kind == 2) {
    for (int h0 = first; h0 < end; h0 += kInFlight) {
      fetch(h0);
#pragma unroll
      for (int n = 0; n < kInFlight; ++n) {
        if (h0 + n >= end) break;                              // the same for the whole wavefront
        float x[8];
        unpack8<DT>(raw[n], x);
        store_word<D, GROUP>(quantize_word<GROUP>(x), slot, w, true, a.sh, a.cache + (h0 + n) * a.sh.record_bytes());
      }
    }
    return;
  }

  // cosines and sines: interleaved, of four pairs; by halves, of eight channels
  const int half = a.rot / 2;
  const bool turned = c < a.rot, low = INTERLEAVED || c < half;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.0f;
    sn[i] = 0.0f;
  }
  if (turned && live) {
    const int64_t p = a.positions[t];
    if (p >= 0 && p < a.table_rows) {
      const f32x4* row = reinterpret_cast<const f32x4*>(a.table + p * a.rot + (INTERLEAVED ? c : 2 * (low ? c : c - half)));
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
        const f32x4 v = row[i];
        cs[2 * i] = v.x;
        sn[2 * i] = low ? (INTERLEAVED ? v.y : -v.y) : v.y;
        cs[2 * i + 1] = v.z;
        sn[2 * i + 1] = low ? (INTERLEAVED ? v.w : -v.w) : v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __builtin_nanf("");
    }
  }
  const bool norm = rows.weight != nullptr;
  const int away = turned && !INTERLEAVED ? (low ? half : -half) : 0;      // channels to the partner's
  const int partner = lane + away / 8;
  float weight[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) weight[i] = 1.0f;
  if (norm) load_weight<DT>(rows.weight, a.w_f32, c, weight);

  if (kind == 0) {
    constexpr float inv_d = 1.0f / D;
    uint16_t* out = rows.out + (t * rows.heads) * D + c;
    for (int h0 = first; h0 < end; h0 += kInFlight) {
      fetch(h0);
#pragma unroll
      for (int n = 0; n < kInFlight; ++n) {
        if (h0 + n >= end) break;
        float x[8];
        unpack8<DT>(raw[n], x);
        if (norm) {
          const float inv = inverse_rms(head_sum_of_squares(x, kLanes), inv_d, a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * weight[i];
        }
        if constexpr (INTERLEAVED) {
          if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = x[2 * i], f = x[2 * i + 1];
              x[2 * i] = fmaf(e, cs[i], -(f * sn[i]));
              x[2 * i + 1] = fmaf(f, cs[i], e * sn[i]);
            }
          }
        } else if (a.rot > 0) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], partner, kWave);
          if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
          }
        }
        if (live)
          st16_nt(out + (h0 + n) * D, u32x4{pack_pair<DT>(x[0], x[1]), pack_pair<DT>(x[2], x[3]),
                                            pack_pair<DT>(x[4], x[5]), pack_pair<DT>(x[6], x[7])});
      }
    }
    return;
  }

  float other[8];                                              // the partner's weights
#pragma unroll
  for (int i = 0; i < 8; ++i) other[i] = 1.0f;
  if (norm && !INTERLEAVED) load_weight<DT>(rows.weight, a.w_f32, c + away, other);
  for (int h0 = first; h0 < end; h0 += kInFlight) {
    fetch(h0);
#pragma unroll
    for (int n = 0; n < kInFlight; ++n) {
      if (h0 + n >= end) break;
      float x[8];
      unpack8<DT>(raw[n], x);
      double inv = 1.0;
      if (norm) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
        sum += dpp_d<kDppXor1>(sum);
        sum += dpp_d<kDppXor2>(sum);
        sum += dpp_d<kDppHalfMirror>(sum);
        if constexpr (kLanes >= 16) sum += dpp_d<kDppMirror>(sum);
        if constexpr (kLanes >= 32) sum += __shfl_xor(sum, 16, kWave);
        inv = inverse_sqrt(fma(sum, 1.0 / D, static_cast<double>(a.eps)));
      }
      float key[8];
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double e = norm ? x[2 * i] * inv * weight[2 * i] : x[2 * i];
          const double f = norm ? x[2 * i + 1] * inv * weight[2 * i + 1] : x[2 * i + 1];
          key[2 * i] = static_cast<float>(turned ? fma(e, static_cast<double>(cs[i]), -(f * sn[i])) : e);
          key[2 * i + 1] = static_cast<float>(turned ? fma(f, static_cast<double>(cs[i]), e * sn[i]) : f);
        }
      } else {
        float y[8];
        u32x4 theirs;
#pragma unroll
        for (int j = 0; j < 4; ++j) theirs[j] = __shfl(raw[n][j], partner, kWave);
        unpack8<DT>(theirs, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double e = norm ? x[i] * inv * weight[i] : x[i];
          const double f = norm ? y[i] * inv * other[i] : y[i];
          key[i] = static_cast<float>(turned ? fma(e, static_cast<double>(cs[i]), f * sn[i]) : e);
        }
      }
      store_word<D, GROUP>(quantize_word<GROUP>(key), slot, w, false, a.sh, a.cache + (h0 + n) * a.sh.record_bytes());
    }
  }
}

// Deals the heads; the launch's grid.
dim3 deal(RopeAppend& a) {
  const int64_t slices = ceil_div(a.T, 512 / a.sh.D);
  const int64_t heads = a.q.heads + 2 * static_cast<int64_t>(a.sh.heads);
  // heads a wavefront takes: as many as leave 12 wavefronts a compute unit.  With a
  // read of what was appended, 1, 2, 4, 8, 16 heads: 512 tokens of 32/8 heads of 128
  // 11.0, 9.2, 10.2, 12.8, 13.1 us; 1024 17.3, 13.9, 12.6, 15.1, 14.4; 8191 112, 78, 60, 64, 50.
  a.per = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, heads * slices / (12 * device_cus()))));
  a.q_parts = static_cast<int>(ceil_div(a.q.heads, a.per));
  a.kv_parts = static_cast<int>(ceil_div(a.sh.heads, a.per));
  return dim3(static_cast<unsigned>(slices), static_cast<unsigned>(ceil_div(a.q_parts + 2 * a.kv_parts, 4)));
}

template <int DT, int D, int GROUP>
void launch_rope_append(const RopeAppend& a, dim3 grid, bool interleaved, hipStream_t s) {
  if (interleaved) kv4_rope_append_kernel<DT, D, GROUP, true><<<grid, 256, 0, s>>>(a);
  else kv4_rope_append_kernel<DT, D, GROUP, false><<<grid, 256, 0, s>>>(a);
}

template <int DT>
void rope_append_shape(const RopeAppend& a, dim3 grid, bool interleaved, hipStream_t s) {
  switch (a.sh.D * 1000 + a.sh.group) {
    case 64032: launch_rope_append<DT, 64, 32>(a, grid, interleaved, s); break;
    case 64064: launch_rope_append<DT, 64, 64>(a, grid, interleaved, s); break;
    case 128032: launch_rope_append<DT, 128, 32>(a, grid, interleaved, s); break;
    case 128064: launch_rope_append<DT, 128, 64>(a, grid, interleaved, s); break;
    case 128128: launch_rope_append<DT, 128, 128>(a, grid, interleaved, s); break;
    case 256032: launch_rope_append<DT, 256, 32>(a, grid, interleaved, s); break;
    case 256064: launch_rope_append<DT, 256, 64>(a, grid, interleaved, s); break;
    default: launch_rope_append<DT, 256, 128>(a, grid, interleaved, s); break;
  }
}

}  // namespace
}  // namespace qmm

extern "C" int kv4_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                               const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                               int64_t v_token_stride, int64_t v_head_stride, int dtype, int64_t T,
                               const int64_t* positions, const float* table, int64_t table_rows, int64_t rot,
                               int interleaved, const void* q_weight, const void* k_weight, int w_dtype, float eps,
                               const int64_t* slots, uint8_t* cache, int64_t pages, int64_t kv_heads, int64_t head_dim,
                               int64_t page, int group, void* q_out, void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!k || !v || !slots || !cache || T < 0 || q_heads < 0 || (q_heads > 0 && (!q || !q_out)) || rot < 0 ||
      dtype < QMM_F32 || dtype > QMM_I32 || !(eps >= 0.0f))
    return QMM_EINVAL;
  if (rot > 0 && (!positions || !table || table_rows <= 0)) return QMM_EINVAL;
  const bool weights = q_weight || k_weight;
  if (weights && (w_dtype < QMM_F32 || w_dtype > QMM_I32)) return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if ((dtype != QMM_BF16 && dtype != QMM_F16) || (weights && w_dtype != dtype && w_dtype != QMM_F32))
    return QMM_EUNSUPPORTED;
  if (rot % 16 != 0 || rot > head_dim) return QMM_EUNSUPPORTED;
  if (q_heads > 65535 || T >= (int64_t{1} << 24)) return QMM_ERANGE;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 8) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(table, 16) ||
      (q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || ((q_token_stride | q_head_stride) & 7))) ||
      ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 7))
    return QMM_EALIGN;
  RopeAppend a{};
  a.q = {static_cast<const uint16_t*>(q), q_token_stride, q_head_stride, q_weight, static_cast<uint16_t*>(q_out),
         static_cast<int32_t>(q_heads)};
  a.k = {static_cast<const uint16_t*>(k), k_token_stride, k_head_stride, k_weight, nullptr, sh.heads};
  a.v = {static_cast<const uint16_t*>(v), v_token_stride, v_head_stride, nullptr, nullptr, sh.heads};
  a.w_f32 = weights && w_dtype == QMM_F32;
  a.positions = positions;
  a.table = table;
  a.table_rows = table_rows;
  a.rot = static_cast<int>(rot);
  a.eps = eps;
  a.slots = slots;
  a.cache = cache;
  a.sh = sh;
  a.T = T;
  const dim3 grid = deal(a);
  if (static_cast<int64_t>(grid.x) * grid.y >= (int64_t{1} << 24)) return QMM_ERANGE;   // blocks of 256 threads a launch holds
  if (dtype == QMM_BF16) rope_append_shape<QMM_BF16>(a, grid, interleaved != 0, as_stream(stream));
  else rope_append_shape<QMM_F16>(a, grid, interleaved != 0, as_stream(stream));
  return launch_status();
}
