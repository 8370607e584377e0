// kv4_attention.hip -- causal attention over the 4-bit paged cache (the
// format and the masks are stated in include/qmm.h).

#include <algorithm>

#include "kv4_device.h"

namespace qmm {
namespace {

struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs, T;
  const int32_t* cu_q;
  const int32_t* context;
  const int32_t* table;
  int64_t table_width, table_stride;
  const uint8_t* cache;
  Kv4Shape sh;
  int q_heads, seqs;
  float scale;
  int64_t window, sinks;
  uint16_t* out;
  float* lse;
};

// One wavefront per query row and head, 64 keys a step: lane l takes key l of
// the step for the scores, channels l, l + 64, .. for the sums.
template <int DT>
__global__ __launch_bounds__(64) void attention_row_kernel(AttnArgs a) {
  const int lane = threadIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  const int kvh = h / (a.q_heads / a.sh.heads);
  const int64_t row0 = a.cu_q ? std::max(0, a.cu_q[b]) : b;
  const int64_t row1 = a.cu_q ? std::min<int64_t>(a.T, a.cu_q[b + 1]) : b + 1;
  const int64_t limit = a.table_width * a.sh.page;
  const int64_t ctx = std::max<int64_t>(0, std::min<int64_t>(a.context[b], limit));
  const int D = a.sh.D, page = a.sh.page;
  __shared__ float qs[256];
  for (int64_t row = row0 + blockIdx.x; row < row1; row += gridDim.x) {
    const int64_t pos = ctx - (row1 - row0) + (row - row0);
    const uint16_t* q = a.q + row * a.q_ts + h * a.q_hs;
    __syncthreads();
    for (int d = lane; d < D; d += 64) qs[d] = DT == QMM_BF16 ? bf16lo_to_f32(q[d]) : f16lo_to_f32(q[d]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t j0 = 0; j0 <= pos; j0 += 64) {
      const int64_t j = j0 + lane;
      int id = -1;
      if (j <= pos) id = a.table[b * a.table_stride + (j >> a.sh.shift)];
      const bool seen = j <= pos && id >= 0 && id < a.sh.pages && (a.window == 0 || j > pos - a.window || j < a.sinks);
      const int t = static_cast<int>(j) & (page - 1);
      const int64_t rec = seen ? (static_cast<int64_t>(id) * a.sh.heads + kvh) * a.sh.record_bytes() : 0;
      float x = -INFINITY;
      if (seen) {
        x = 0.0f;
        for (int w = 0; w < D / 8; ++w) {
          const uint32_t word = *reinterpret_cast<const uint32_t*>(a.cache + rec + kv4_k_word(t, w, D));
          const uint32_t param =
              reinterpret_cast<const uint32_t*>(a.cache + rec + a.sh.k_params())[8 * w / a.sh.group * page + t];
          const float s = kv4_scale(param), z = kv4_zero(param);
          for (int e = 0; e < 8; ++e) x = fmaf(qs[8 * w + e], (static_cast<float>(kv4_code(word, e)) - z) * s, x);
        }
        x *= a.scale;
      }
      const float m_new = fmaxf(m, wave_max(x));
      const float base = m_new == -INFINITY ? 0.0f : m_new;
      const float p = expf(x - base), fade = expf(m - base);
      m = m_new;
      l = l * fade + wave_sum(p);
      for (int i = 0; i < 4; ++i) o[i] *= fade;
      for (int s = 0; s < 64; ++s) {
        if (!__shfl(static_cast<int>(seen), s, kWave)) continue;
        const float ps = __shfl(p, s, kWave);
        const int64_t rs = __shfl(rec, s, kWave);
        const int ts = __shfl(t, s, kWave);
        for (int i = 0; i < 4; ++i) {
          const int d = lane + 64 * i;
          if (d >= D) break;
          const uint32_t word = *reinterpret_cast<const uint32_t*>(a.cache + rs + kv4_v_word(ts, d >> 3, D, page));
          const uint32_t param =
              reinterpret_cast<const uint32_t*>(a.cache + rs + a.sh.v_params())[d / a.sh.group * page + ts];
          o[i] = fmaf(ps, (static_cast<float>(kv4_code(word, d & 7)) - kv4_zero(param)) * kv4_scale(param), o[i]);
        }
      }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int i = 0; i < 4 && lane + 64 * i < D; ++i)
      a.out[(row * a.q_heads + h) * D + lane + 64 * i] = static_cast<uint16_t>(pack2<DT>(o[i] * inv, 0.0f));
    if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
  }
}

}  // namespace
}  // namespace qmm

extern "C" size_t kv4_attention_workspace_bytes(int64_t T, int64_t seqs, int64_t max_q, int64_t q_heads,
                                                int64_t kv_heads, int64_t head_dim, int64_t max_context,
                                                int64_t window, int64_t sinks) {
  return 0;
}

extern "C" int kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, int64_t T,
                             int64_t q_heads, const int32_t* cu_q, int64_t seqs, int64_t max_q,
                             const int32_t* context, const int32_t* page_table, int64_t table_width,
                             int64_t table_stride, const uint8_t* cache, int64_t pages, int64_t kv_heads,
                             int64_t head_dim, int64_t page, int group, float scale, int64_t window, int64_t sinks,
                             void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (T == 0 || seqs == 0) return T == 0 ? QMM_OK : QMM_EINVAL;
  if (!q || !context || !page_table || !cache || !out || T < 0 || seqs < 0 || q_heads <= 0 || max_q <= 0 ||
      table_width <= 0 || table_stride < table_width || window < 0 || sinks < 0 || !(scale == scale) ||
      dtype < QMM_F32 || dtype > QMM_I32 || (!cu_q && T != seqs))
    return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (q_heads % kv_heads != 0) return QMM_EINVAL;
  if (dtype != QMM_BF16 && dtype != QMM_F16) return QMM_EUNSUPPORTED;
  if (T >= (int64_t{1} << 31) || seqs > 65535 || q_heads > 65535 || table_width * page >= (int64_t{1} << 31))
    return QMM_ERANGE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16) || !aligned(lse, 4) || !aligned(context, 4) ||
      !aligned(cu_q, 4) || !aligned(page_table, 4) || ((q_token_stride | q_head_stride) & 7))
    return QMM_EALIGN;
  AttnArgs a{static_cast<const uint16_t*>(q), q_token_stride, q_head_stride, T, cu_q, context, page_table,
             table_width, table_stride, cache, sh, static_cast<int>(q_heads), static_cast<int>(seqs), scale, window,
             sinks, static_cast<uint16_t*>(out), lse};
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(cu_q ? max_q : 1, 65535)), static_cast<unsigned>(q_heads),
                  static_cast<unsigned>(seqs));
  if (dtype == QMM_BF16)
    attention_row_kernel<QMM_BF16><<<grid, 64, 0, as_stream(stream)>>>(a);
  else
    attention_row_kernel<QMM_F16><<<grid, 64, 0, as_stream(stream)>>>(a);
  return launch_status();
}
