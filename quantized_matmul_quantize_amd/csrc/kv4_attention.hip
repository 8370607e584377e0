// kv4_attention.hip -- entry points of the attention over the 4-bit paged
// cache: argument checks and the launch plan (kernels: kv4_attention.h).

#include <algorithm>

#include "kv4_attention_args.h"

namespace qmm {
namespace {

constexpr int64_t kLeastSteps = 24;     // of a block whose sequence is split

// How the work is cut.  Up to 96 rows the wavefronts of a block share the rows
// and split the keys; beyond, each has rows of its own, of shared operands
// (32 sequences of 4000 tokens, 8 kv heads, D 128 in one group, us: 64 rows
// 74 shared, 130 own; 96 rows 110, 137; 128 rows 136, 148; 256 rows 259, 185;
// in groups of 64: 96 rows 140, 160; 128 rows 172, 160; 256 rows 329, 313).
// The fewer the rows, the more steps a wavefront takes at once; where a tile
// for every 8 rows leaves the chip three quarters empty (half, where the keys
// are too few to be split over blocks), blocks of 8 rows in pairs of steps are
// the better ones, where one for every 16 leaves it not full, those of 16 are
// (us, D 128 in groups of 64, 8 kv heads, 16 rows: 8 sequences of 2000 tokens
// 17.9 in tiles of 8, 20.3 of 16, 16 of 1000 14.3 and 16.3, 16 of 2000 26.3
// and 23.7, 32 of 4000 51 and 46; 20 rows: 4 of 2000 18.1 and 20.1, 8 of 2000
// 24.0 and 21.2, there in tiles of 32 29.0; 32 of 4000 in tiles of 16 and of
// 32: 20 rows 67 and 64, 48 rows 81 and 91, 64 rows 106 and 91).
// Keys are split over blocks only where rows and heads leave compute units idle.
AttnPlan plan_of(int64_t seqs, int64_t max_q, int64_t ratio, int64_t kv_heads, int64_t D, int group,
                 int64_t max_context, int64_t window, int64_t sinks) {
  AttnPlan p{};
  p.max_q = max_q;
  const int64_t rows = max_q * ratio, fill = 2 * device_cus();
  p.ws = rows <= 96;
  const int64_t kept = std::min(window, max_context) + std::min(sinks, max_context);
  const int64_t keys = window > 0 ? std::min(max_context, kept) : max_context;
  const bool whole = keys < 2 * kLeastSteps * kStep;
  const bool eights = rows <= 8 || (p.ws && (whole ? 2 : 4) * seqs * kv_heads * ceil_div(rows, 8) <= fill);
  const bool sixteens = eights || rows <= 16 || seqs * kv_heads * ceil_div(rows, 16) < fill;
  p.pk = eights && attention_pairs(static_cast<int>(D), group) ? 2 : 1;
  p.nt = !p.ws ? attention_chunk_tiles(static_cast<int>(D), group)
               : sixteens ? 1 : attention_tiles(static_cast<int>(D), group);
  p.rows = 16 / p.pk * p.nt * (p.ws ? 1 : kWaves);
  // (blocks loop over row tiles past these: a launch holds 2^24 blocks of 256 threads)
  p.row_tiles = std::min(ceil_div(rows, p.rows), std::max<int64_t>(1, (int64_t{1} << 22) / (seqs * kv_heads)));
  int64_t steps = ceil_div(max_context, kStep);
  if (window > 0)
    steps = std::min(steps, ceil_div(std::min(window, max_context) + p.rows / ratio + 1, kStep) + 1 +
                                ceil_div(std::min(sinks, max_context), kStep));
  // Two blocks a compute unit, and no fewer than kLeastSteps each: the join of
  // the chunks is a launch of its own (one sequence of 700 tokens: 11.6 us a
  // call whole, 14.3 in three; in a captured graph 11.4 and 11.0), and ragged
  // contexts even out less in larger ones (7 sequences of up to 2301: 29 us in
  // two chunks, 24 in three, 31 in four; two of 131072: 76 us in 16, 65 in 32,
  // 72 in 57).
  const int64_t blocks = seqs * kv_heads * p.row_tiles;
  const int64_t want =
      4 * blocks >= 3 * fill ? 1 : std::max<int64_t>(1, std::min(ceil_div(fill, blocks), steps / kLeastSteps));
  const int64_t round = p.ws ? kWaves * p.pk : 8;         // steps of a round of the wavefronts, or two of a block
  p.chunk = want == 1 ? std::max<int64_t>(steps, 1)
                      : std::max<int64_t>(1, (ceil_div(steps, want) + round / 2) / round) * round;
  p.splits = std::max<int64_t>(1, ceil_div(steps, p.chunk));
  p.blocks = blocks * p.splits;
  return p;
}

size_t workspace_bytes_of(const AttnPlan& p, int64_t T, int64_t q_heads, int64_t D) {
  return p.splits > 1 ? static_cast<size_t>(T) * q_heads * p.splits * (D + 2) * 4 : 0;
}

}  // namespace
}  // namespace qmm

extern "C" size_t kv4_attention_workspace_bytes(int64_t T, int64_t seqs, int64_t max_q, int64_t q_heads,
                                                int64_t kv_heads, int64_t head_dim, int group,
                                                int64_t max_context, int64_t window, int64_t sinks) {
  using namespace qmm;
  if (T <= 0 || seqs <= 0 || max_q <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 ||
      group <= 0 || max_context <= 0 || max_context >= (int64_t{1} << 31) || window < 0 || sinks < 0 || T >= (int64_t{1} << 31) ||
      seqs > 65535 || q_heads > 65535)
    return 0;
  return workspace_bytes_of(plan_of(seqs, std::min(max_q, T), q_heads / kv_heads, kv_heads, head_dim, group,
                                    max_context, window, sinks), T, q_heads, head_dim);
}

extern "C" int kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, int64_t T,
                             int64_t q_heads, const int32_t* cu_q, int64_t seqs, int64_t max_q,
                             const int32_t* context, const int32_t* page_table, int64_t table_width,
                             int64_t table_stride, const uint8_t* cache, int64_t pages, int64_t kv_heads,
                             int64_t head_dim, int64_t page, int group, float scale, int64_t window, int64_t sinks,
                             void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!q || !context || !page_table || !cache || !out || T < 0 || seqs <= 0 || q_heads <= 0 || max_q <= 0 ||
      table_width <= 0 || table_stride < table_width || window < 0 || sinks < 0 || !(scale == scale) ||
      dtype < QMM_F32 || dtype > QMM_I32 || (!cu_q && T != seqs))
    return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (q_heads % kv_heads != 0) return QMM_EINVAL;
  if (dtype != QMM_BF16 && dtype != QMM_F16) return QMM_EUNSUPPORTED;
  if (T >= (int64_t{1} << 31) || T * q_heads >= (int64_t{1} << 31) || seqs > 65535 || q_heads > 65535 ||
      table_width >= (int64_t{1} << 31) || table_width * page > (int64_t{1} << 30))
    return QMM_ERANGE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16) || !aligned(lse, 4) || !aligned(context, 4) ||
      !aligned(cu_q, 4) || !aligned(page_table, 4) || ((q_token_stride | q_head_stride) & 7))
    return QMM_EALIGN;
  const int64_t ratio = q_heads / kv_heads, tokens = table_width * page;
  const AttnPlan p = plan_of(seqs, std::min(max_q, T), ratio, kv_heads, head_dim, group, tokens,
                             window, sinks);
  const size_t need = workspace_bytes_of(p, T, q_heads, head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QMM_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QMM_EALIGN;
  if (p.blocks >= (int64_t{1} << 24)) return QMM_ERANGE;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.cu_q = cu_q;
  a.context = context;
  a.table = page_table;
  a.table_stride = table_stride;
  a.cache = cache;
  a.sh = sh;
  a.T = static_cast<int32_t>(T);
  a.q_heads = static_cast<int32_t>(q_heads);
  a.ratio = static_cast<int32_t>(ratio);
  a.seqs = static_cast<int32_t>(seqs);
  a.limit = static_cast<int32_t>(tokens);
  a.window = static_cast<int32_t>(std::min<int64_t>(window, int64_t{1} << 30));
  a.sinks = static_cast<int32_t>(std::min<int64_t>(sinks, int64_t{1} << 30));
  a.scale_log2 = scale * 1.44269504088896341f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.splits = static_cast<int32_t>(p.splits);
  a.chunk = static_cast<int32_t>(p.chunk);
  a.row_tiles = static_cast<int32_t>(p.row_tiles);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (need > 0 ? T * q_heads * p.splits * head_dim : 0));
  if (dtype == QMM_BF16) attention_bf16(a, p, as_stream(stream));
  else attention_f16(a, p, as_stream(stream));
  return launch_status();
}
