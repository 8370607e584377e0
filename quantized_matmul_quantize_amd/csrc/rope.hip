// rope.hip -- norms of queries and keys for each head with the rotation by
// position in the same pass, and the table of cosines and sines it reads.

#include "qmm_device.h"

namespace qmm {
namespace {

// Angles and functions in fp64: the rounding of p f to fp32 alone would be an
// error of 2^-7 radian at p = 131072.
struct Frequencies {
  double f[256];
};
__global__ __launch_bounds__(256) void rope_table_kernel(Frequencies freq, int half, int64_t rows, double m,
                                                         float2* __restrict__ table) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows * half) return;
  double s, c;
  sincos(static_cast<double>(i / half) * freq.f[i % half], &s, &c);
  table[i] = make_float2(static_cast<float>(m * c), static_cast<float>(m * s));
}

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

// A head's D channels lie on `lanes` (a power of two) consecutive lanes,
// eight channels each.  Bound by memory: 2 bytes read and 2 written per
// channel, 4 rot bytes of table per token.
template <int DT, int WDT>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(HeadRows q, HeadRows k, int64_t T, int D,
                                                           const int64_t* __restrict__ positions,
                                                           const float* __restrict__ table, int64_t table_rows,
                                                           int rot, int interleaved, float eps, int lanes_log2) {
  const int lanes = 1 << lanes_log2;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> lanes_log2;
  const int c = (threadIdx.x & (lanes - 1)) * 8;                // first channel of this lane
  const int heads = q.heads + k.heads;
  const int64_t t = unit / heads;
  const int h = static_cast<int>(unit % heads);
  const bool live = t < T && c < D;
  const HeadRows& r = h < q.heads ? q : k;
  const int hr = h < q.heads ? h : h - q.heads;
  float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (live) load8<DT>(r.in, t * r.token_stride + hr * r.head_stride + c, x);
  if (r.weight) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor(sum, o, kWave);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(D) + eps);
    float w[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (live) load8<WDT>(r.weight, c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
  if (rot > 0) {
    const int half = rot / 2;
    int64_t p = live ? positions[t] : 0;
    const bool known = p >= 0 && p < table_rows;
    const float2* row = reinterpret_cast<const float2*>(table) + (known ? p : 0) * half;
    if (interleaved) {
      if (live && c < rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = row[c / 2 + i];
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = known ? a * cs.x - b * cs.y : __builtin_nanf("");
          x[2 * i + 1] = known ? b * cs.x + a * cs.y : __builtin_nanf("");
        }
      }
    } else {
      // the partner's eight channels are half a rotation away, on another lane
      const bool low = c < half;
      const int partner = (threadIdx.x & (kWave - 1)) + (c < rot ? (low ? half / 8 : -(half / 8)) : 0);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], partner, kWave);
      if (live && c < rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 cs = row[(low ? c : c - half) + i];
          const float turned = low ? x[i] * cs.x - y[i] * cs.y : x[i] * cs.x + y[i] * cs.y;
          x[i] = known ? turned : __builtin_nanf("");
        }
      }
    }
  }
  if (!live) return;
  uint16_t* o = r.out + (t * r.heads + hr) * D + c;
  *reinterpret_cast<u32x4*>(o) =
      u32x4{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7])};
}

}  // namespace
}  // namespace qmm

extern "C" int rope_table(const double* inv_freq, int64_t half, int64_t rows, double m, float* table, void* stream) {
  using namespace qmm;
  if (!inv_freq || !table || half <= 0 || rows <= 0) return QMM_EINVAL;
  if (half > 256) return QMM_EUNSUPPORTED;
  if (rows >= (int64_t{1} << 31)) return QMM_ERANGE;
  if (!aligned(table, 16)) return QMM_EALIGN;
  Frequencies f = {};
  for (int64_t i = 0; i < half; ++i) f.f[i] = inv_freq[i];
  rope_table_kernel<<<static_cast<unsigned>(ceil_div(rows * half, 256)), 256, 0, as_stream(stream)>>>(
      f, static_cast<int>(half), rows, m, reinterpret_cast<float2*>(table));
  return launch_status();
}

extern "C" int qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                            const void* k, int64_t k_token_stride, int64_t k_head_stride, int64_t k_heads, int dtype,
                            int64_t T, int64_t head_dim, const int64_t* positions, const float* table,
                            int64_t table_rows, int64_t rot, int interleaved, const void* q_weight,
                            const void* k_weight, int w_dtype, float eps, void* q_out, void* k_out, void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!q || !q_out || q_heads <= 0 || k_heads < 0 || (k_heads > 0 && (!k || !k_out)) || T < 0 || head_dim <= 0 ||
      rot < 0 || dtype < QMM_F32 || dtype > QMM_I32 || !(eps >= 0.0f))
    return QMM_EINVAL;
  if (rot > 0 && (!positions || !table || table_rows <= 0)) return QMM_EINVAL;
  const bool weights = q_weight || k_weight;
  if (weights && (w_dtype < QMM_F32 || w_dtype > QMM_I32)) return QMM_EINVAL;
  if ((dtype != QMM_BF16 && dtype != QMM_F16) || (weights && w_dtype != dtype && w_dtype != QMM_F32))
    return QMM_EUNSUPPORTED;
  if (head_dim % 8 != 0 || head_dim > 512 || rot % 16 != 0 || rot > head_dim) return QMM_EUNSUPPORTED;
  if (q_heads > 65535 || k_heads > 65535) return QMM_ERANGE;
  int lanes_log2 = 0;
  while ((8 << lanes_log2) < head_dim) ++lanes_log2;
  const int64_t units = T < (int64_t{1} << 31) ? T * (q_heads + k_heads) : (int64_t{1} << 62);
  const int64_t blocks = ceil_div(units, 256 >> lanes_log2);
  if (blocks >= (int64_t{1} << 31)) return QMM_ERANGE;
  if (!aligned(q, 16) || !aligned(q_out, 16) || (k_heads > 0 && (!aligned(k, 16) || !aligned(k_out, 16))) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(table, 16) ||
      ((q_token_stride | q_head_stride) & 7) || (k_heads > 0 && ((k_token_stride | k_head_stride) & 7)))
    return QMM_EALIGN;
  const HeadRows qr{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride, q_weight,
                    static_cast<uint16_t*>(q_out), static_cast<int32_t>(q_heads)};
  const HeadRows kr{static_cast<const uint16_t*>(k), k_token_stride, k_head_stride, k_weight,
                    static_cast<uint16_t*>(k_out), static_cast<int32_t>(k_heads)};
  const unsigned grid = static_cast<unsigned>(blocks);
  const int D = static_cast<int>(head_dim), r = static_cast<int>(rot);
  hipStream_t s = as_stream(stream);
  const bool f32w = w_dtype == QMM_F32;
#define QMM_LAUNCH(DT, WDT) \
  qk_norm_rope_kernel<DT, WDT><<<grid, 256, 0, s>>>(qr, kr, T, D, positions, table, table_rows, r, interleaved != 0, \
                                                    eps, lanes_log2)
  if (dtype == QMM_BF16) {
    if (f32w) QMM_LAUNCH(QMM_BF16, QMM_F32); else QMM_LAUNCH(QMM_BF16, QMM_BF16);
  } else {
    if (f32w) QMM_LAUNCH(QMM_F16, QMM_F32); else QMM_LAUNCH(QMM_F16, QMM_F16);
  }
#undef QMM_LAUNCH
  return launch_status();
}
