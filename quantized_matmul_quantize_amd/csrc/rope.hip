// rope.hip -- norms of queries and keys for each head with the rotation by
// position in the same pass, and the table of cosines and sines it reads.

#include <algorithm>

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
// eight channels each; a block takes one token (blockIdx.x) and `per_block`
// of its heads (blockIdx.y), kHeads passes at a time in flight: the cosines,
// sines and weights of a lane's channels are loaded once for all of them.
// Bound by memory: 2 bytes read and 2 written per channel, 4 rot bytes of
// table per token; 8191 tokens of 64 and 8 heads of 128, 64 channels rotated,
// not cached, 58 us, 5.2 TB/s, the rate of a large copy.
constexpr int kHeads = 4;

template <int DT, int WDT, bool NORM, bool INTERLEAVED>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(HeadRows q, HeadRows k, int D,
                                                           const int64_t* __restrict__ positions,
                                                           const float* __restrict__ table, int64_t table_rows,
                                                           int rot, float eps, int lanes_log2, int per_block) {
  const int lanes = 1 << lanes_log2, width = 256 >> lanes_log2;
  const int c = (threadIdx.x & (lanes - 1)) * 8;                // first channel of this lane
  const int64_t t = blockIdx.x;
  const int heads = q.heads + k.heads;
  const int first = static_cast<int>(blockIdx.y) * per_block + (static_cast<int>(threadIdx.x) >> lanes_log2);
  const int end = min(static_cast<int>(blockIdx.y + 1) * per_block, heads);
  const bool live = c < D, turned = c < rot;
  const int half = rot / 2;
  const bool low = INTERLEAVED || c < half;

  float cs[8], sn[8];      // interleaved: four pairs; halves: eight, the sine negated in the first half
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.0f;
    sn[i] = 0.0f;
  }
  if (rot > 0 && turned) {
    const int64_t p = positions[t];
    if (p >= 0 && p < table_rows) {
      const f32x4* row = reinterpret_cast<const f32x4*>(table + p * rot + (INTERLEAVED ? c : 2 * (low ? c : c - half)));
#pragma unroll
      for (int i = 0; i < (INTERLEAVED ? 2 : 4); ++i) {
        const f32x4 v = row[i];
        cs[2 * i] = v.x;
        sn[2 * i] = INTERLEAVED || !low ? v.y : -v.y;
        cs[2 * i + 1] = v.z;
        sn[2 * i + 1] = INTERLEAVED || !low ? v.w : -v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __builtin_nanf("");
    }
  }
  float qw[8], kw[8];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) qw[i] = kw[i] = 0.0f;
    if (live && q.weight) load8<WDT>(q.weight, c, qw);
    if (live && k.weight) load8<WDT>(k.weight, c, kw);
  }
  // the partner's eight channels are half a rotation away, on another lane of the head
  const int partner = (threadIdx.x & (kWave - 1)) + (turned ? (low ? half / 8 : -(half / 8)) : 0);
  const float inv_d = 1.0f / static_cast<float>(D);

  for (int h0 = first; h0 < end; h0 += kHeads * width) {
    u32x4 raw[kHeads];
#pragma unroll
    for (int n = 0; n < kHeads; ++n) {
      const int h = h0 + n * width;
      raw[n] = u32x4{0u, 0u, 0u, 0u};
      if (live && h < end) {
        const HeadRows& r = h < q.heads ? q : k;
        raw[n] = ld16_nt(r.in + t * r.token_stride + (h < q.heads ? h : h - q.heads) * r.head_stride + c);
      }
    }
#pragma unroll
    for (int n = 0; n < kHeads; ++n) {
      const int h = h0 + n * width;
      if (h0 - first + n * width >= per_block) break;           // the same for the whole block
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = DT == QMM_BF16 ? bf16lo_to_f32(raw[n][j]) : f16lo_to_f32(raw[n][j]);
        x[2 * j + 1] = DT == QMM_BF16 ? bf16hi_to_f32(raw[n][j]) : f16hi_to_f32(raw[n][j]);
      }
      const bool is_q = h < q.heads;
      if constexpr (NORM) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
        if (lanes >= 2) sum += dpp_f<kDppXor1>(sum);
        if (lanes >= 4) sum += dpp_f<kDppXor2>(sum);
        if (lanes >= 8) sum += dpp_f<kDppHalfMirror>(sum);
        if (lanes >= 16) sum += dpp_f<kDppMirror>(sum);
        if (lanes >= 32) sum += __shfl_xor(sum, 16, kWave);
        if (lanes >= 64) sum += __shfl_xor(sum, 32, kWave);
        if (is_q ? q.weight != nullptr : k.weight != nullptr) {
          // the instruction takes subnormal numbers for 0
          const float mean = fmaf(sum, inv_d, eps);
          const bool tiny = mean < 0x1p-126f;
          const float inv = __builtin_amdgcn_rsqf(tiny ? mean * 0x1p64f : mean) * (tiny ? 0x1p32f : 1.0f);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (is_q ? qw[i] : kw[i]);
        }
      }
      if (rot > 0) {
        if constexpr (INTERLEAVED) {
          if (turned) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[2 * i], b = x[2 * i + 1];
              x[2 * i] = fmaf(a, cs[i], -(b * sn[i]));
              x[2 * i + 1] = fmaf(b, cs[i], a * sn[i]);
            }
          }
        } else {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], partner, kWave);
          if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], y[i] * sn[i]);
          }
        }
      }
      if (!live || h >= end) continue;
      uint16_t* o = is_q ? q.out + (t * q.heads + h) * D + c : k.out + (t * k.heads + h - q.heads) * D + c;
      st16_nt(o, u32x4{pack_pair<DT>(x[0], x[1]), pack_pair<DT>(x[2], x[3]), pack_pair<DT>(x[4], x[5]), pack_pair<DT>(x[6], x[7])});
    }
  }
}

template <int DT, int WDT>
void launch_rope(const HeadRows& q, const HeadRows& k, int64_t T, int D, const int64_t* positions, const float* table,
                 int64_t rows, int rot, bool interleaved, float eps, int lanes_log2, hipStream_t s) {
  const int heads = q.heads + k.heads, width = 256 >> lanes_log2;
  // Heads of a block: all, but for few tokens as many blocks as fill the chip
  // (32 and 8 heads of 128, all and fewest heads a block in us: 1 token 4.4,
  // 3.0; 256 tokens 4.8, 4.2; 1024 9.0, 10.7; 8192 46, 66).
  const int64_t passes = ceil_div(heads, width);
  const int64_t split = std::min<int64_t>(passes, ceil_div(4 * device_cus(), T));
  const int per_block = static_cast<int>(ceil_div(passes, split) * width);
  const dim3 grid(static_cast<unsigned>(T), static_cast<unsigned>(ceil_div(heads, per_block)));
  const bool norm = q.weight || k.weight;
#define QMM_ROPE(NORM, INTER) \
  qk_norm_rope_kernel<DT, WDT, NORM, INTER><<<grid, 256, 0, s>>>(q, k, D, positions, table, rows, rot, eps, lanes_log2, \
                                                                 per_block)
  if (norm) {
    if (interleaved) QMM_ROPE(true, true); else QMM_ROPE(true, false);
  } else {
    if (interleaved) QMM_ROPE(false, true); else QMM_ROPE(false, false);
  }
#undef QMM_ROPE
}

}  // namespace
}  // namespace qmm

extern "C" int rope_table(const double* inv_freq, int64_t half, int64_t rows, double m, float* table, void* stream) {
  using namespace qmm;
  if (!inv_freq || !table || half <= 0 || rows <= 0) return QMM_EINVAL;
  if (half > 256) return QMM_EUNSUPPORTED;
  if (rows >= (int64_t{1} << 31) / half) return QMM_ERANGE;      // a launch holds 2^24 blocks of 256 threads
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
  if (T >= (int64_t{1} << 24)) return QMM_ERANGE;                // blocks of 256 threads a launch holds
  if (!aligned(q, 16) || !aligned(q_out, 16) || (k_heads > 0 && (!aligned(k, 16) || !aligned(k_out, 16))) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 8) || !aligned(table, 16) ||
      ((q_token_stride | q_head_stride) & 7) || (k_heads > 0 && ((k_token_stride | k_head_stride) & 7)))
    return QMM_EALIGN;
  const HeadRows qr{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride, q_weight,
                    static_cast<uint16_t*>(q_out), static_cast<int32_t>(q_heads)};
  const HeadRows kr{static_cast<const uint16_t*>(k), k_token_stride, k_head_stride, k_weight,
                    static_cast<uint16_t*>(k_out), static_cast<int32_t>(k_heads)};
  const int D = static_cast<int>(head_dim), r = static_cast<int>(rot);
  hipStream_t s = as_stream(stream);
  const bool f32w = weights && w_dtype == QMM_F32, inter = interleaved != 0;
  if (dtype == QMM_BF16) {
    if (f32w) launch_rope<QMM_BF16, QMM_F32>(qr, kr, T, D, positions, table, table_rows, r, inter, eps, lanes_log2, s);
    else launch_rope<QMM_BF16, QMM_BF16>(qr, kr, T, D, positions, table, table_rows, r, inter, eps, lanes_log2, s);
  } else {
    if (f32w) launch_rope<QMM_F16, QMM_F32>(qr, kr, T, D, positions, table, table_rows, r, inter, eps, lanes_log2, s);
    else launch_rope<QMM_F16, QMM_F16>(qr, kr, T, D, positions, table, table_rows, r, inter, eps, lanes_log2, s);
  }
  return launch_status();
}
