// kv4_prefix.hip -- entry points of the attention of a batch in groups that share
// a prefix: argument checks and the launch plan (kernels: kv4_attention.h,
// kv4_attention_chunk.h for own parts, kv4_attention_rows.h for prefixes).
//
// A prefix is a part of its own: attended to for a group with all of its rows, in
// tiles of 8, 16, 32 or up to 256 that read it once each, which turns loads and
// expansions of codes per sequence into matrix products, and joined with each
// sequence's own part by log-sum-exp in fp32.
// Two launches where both parts take the kernel for few rows, else three.  24
// questions on each of two documents of 100000 tokens (64/8 heads of 128) 240
// us, 4 beams after 1000 tokens (32/8) 13.5.

#include <algorithm>

#include "kv4_attention_args.h"

namespace qmm {
namespace {

// The least steps of a chunk.  Chunks are joined in any case, so they are
// smaller than where a split would cost the join.
constexpr int64_t kLeastSteps = 8;

// How a part is cut: `items` (groups, or sequences) of up to `rows` rows and
// `keys` keys.  Which kernel: by rows, as for a batch without prefixes, unless
// `pk` steps at once of 16 rows are asked for.
AttnPlan part_plan(bool prefix, int64_t items, int64_t rows, int64_t kv_heads, int64_t D, int group, int64_t keys,
                   int64_t* round, int pk = 0) {
  AttnPlan p{};
  const int d = static_cast<int>(D);
  const int64_t steps = std::max<int64_t>(1, ceil_div(keys, kStep));
  // The kernel for many rows starts later, leaves more to join and shares no launch
  // with the own parts: prefixes of few steps (of 16 rows, for each of the blocks
  // at once) stay with the kernel for few.  256 rows in 8 heads of 128 after 4096
  // tokens (32 steps) 48 us by rows, 30 here; 8192 50 and 40; 12288 54 and 52;
  // 16384 59 and 64.  216 rows of 12 prefixes in 2 heads of 64 after 1500 tokens (31)
  // 40 and 30; 3000 42.5 and 44.  256 rows of 256 after 4096 (32) 62 and 54; 8192 73 both.
  const int64_t short_of = (D == 128 ? 96 : 48) * 2 * device_cus();
  p.ws = rows <= 96 || (prefix && items * kv_heads * ceil_div(rows, 16) * steps <= short_of);
  const int64_t fill = (p.ws || !prefix ? 2 : 1) * device_cus();
  const bool eights = rows <= 8;
  const bool sixteens = eights || rows <= 16 || items * kv_heads * ceil_div(rows, 16) < fill;
  p.pk = pk ? pk : eights && attention_pairs(d, group) ? 2 : 1;
  p.nt = !p.ws ? attention_chunk_tiles(d, group) : sixteens || pk ? 1 : attention_tiles(d, group);
  p.rows = p.ws ? 16 / p.pk * p.nt : prefix ? (D == 256 ? 128 : 256) : 16 * p.nt * kWaves;
  // (blocks loop over row tiles past these: a launch holds 2^24 blocks of 256 threads)
  p.row_tiles = std::min(ceil_div(rows, p.rows), std::max<int64_t>(1, (int64_t{1} << 22) / (items * kv_heads)));
  const int64_t blocks = items * kv_heads * p.row_tiles;
  *round = p.ws ? kWaves * p.pk : D == 256 ? 1 : 2;
  p.splits = std::max<int64_t>(1, std::min(fill / blocks, steps / std::max(kLeastSteps, *round)));
  p.blocks = blocks * p.splits;
  if (!p.ws && prefix) p.blocks = ceil_div(items * kv_heads * p.splits, 8) * 8 * p.row_tiles;
  return p;
}

struct Plans {
  AttnPlan prefix, own;
  int64_t p_round, round;
  bool together;      // both in one launch
};
Plans plans_of(int64_t seqs, int64_t max_q, int64_t n_groups, int64_t max_group, int64_t max_prefix, int64_t max_tail,
               int64_t ratio, int64_t kv_heads, int64_t D, int group, int64_t tokens, int64_t T) {
  Plans p{};
  max_q = std::min(max_q, T);
  const int64_t rows = std::min(std::min(max_group, seqs) * max_q, T) * ratio;
  p.prefix = part_plan(true, n_groups, rows, kv_heads, D, group, std::min(max_prefix, tokens), &p.p_round);
  p.own = part_plan(false, seqs, max_q * ratio, kv_heads, D, group, std::min(max_tail, tokens), &p.round);
  p.own.max_q = max_q;
  // Kernels of few rows run in one launch, the own parts by the prefix's number of
  // steps at once: 4 beams after 1000 tokens 21 us in two launches, 13.5 in one; 64
  // samples after 4096 tokens 39 and 30; 30000 tokens of 4 beams 32 and 24.
  if (p.prefix.ws && p.own.ws) {
    p.own = part_plan(false, seqs, max_q * ratio, kv_heads, D, group, std::min(max_tail, tokens), &p.round, p.prefix.pk);
    p.own.max_q = max_q;
    p.together = true;
  }
  return p;
}
size_t bytes_of(const Plans& p, int64_t T, int64_t q_heads, int64_t D) {
  return static_cast<size_t>(T) * q_heads * (p.prefix.splits + p.own.splits) * (D + 2) * 4;
}

}  // namespace
}  // namespace qmm

extern "C" size_t kv4_prefix_attention_workspace_bytes(int64_t T, int64_t seqs, int64_t max_q, int64_t n_groups,
                                                       int64_t max_group, int64_t max_prefix, int64_t max_tail,
                                                       int64_t q_heads, int64_t kv_heads, int64_t head_dim, int group,
                                                       int64_t max_context) {
  using namespace qmm;
  if (T <= 0 || seqs <= 0 || max_q <= 0 || n_groups <= 0 || max_group <= 0 || max_prefix <= 0 || max_tail <= 0 ||
      q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 || group <= 0 || max_context <= 0 ||
      max_context >= (int64_t{1} << 31) || T >= (int64_t{1} << 31) || seqs > 65535 || n_groups > 65535 || q_heads > 65535)
    return 0;
  return bytes_of(plans_of(seqs, max_q, n_groups, max_group, max_prefix, max_tail, q_heads / kv_heads, kv_heads,
                           head_dim, group, max_context, T), T, q_heads, head_dim);
}

extern "C" int kv4_prefix_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int dtype, int64_t T,
                                    int64_t q_heads, const int32_t* cu_q, int64_t seqs, int64_t max_q,
                                    const int32_t* context, const int32_t* page_table, int64_t table_width,
                                    int64_t table_stride, const int32_t* groups, const int32_t* prefix,
                                    int64_t n_groups, int64_t max_group, int64_t max_prefix, int64_t max_tail,
                                    const uint8_t* cache, int64_t pages, int64_t kv_heads, int64_t head_dim,
                                    int64_t page, int group, float scale, void* out, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (T == 0) return QMM_OK;
  if (!q || !context || !page_table || !groups || !prefix || !cache || !out || T < 0 || seqs <= 0 || q_heads <= 0 ||
      max_q <= 0 || n_groups <= 0 || max_group <= 0 || max_prefix <= 0 || max_tail <= 0 || table_width <= 0 ||
      table_stride < table_width || !(scale == scale) || dtype < QMM_F32 || dtype > QMM_I32 || (!cu_q && T != seqs))
    return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (q_heads % kv_heads != 0) return QMM_EINVAL;
  if (dtype != QMM_BF16 && dtype != QMM_F16) return QMM_EUNSUPPORTED;
  if (T >= (int64_t{1} << 31) || T * q_heads >= (int64_t{1} << 31) || seqs > 65535 || n_groups > 65535 ||
      q_heads > 65535 || table_width >= (int64_t{1} << 31) || table_width * page > (int64_t{1} << 30))
    return QMM_ERANGE;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(cache, 16) || !aligned(lse, 4) || !aligned(context, 4) ||
      !aligned(cu_q, 4) || !aligned(page_table, 4) || !aligned(groups, 4) || !aligned(prefix, 4) ||
      ((q_token_stride | q_head_stride) & 7))
    return QMM_EALIGN;
  const int64_t ratio = q_heads / kv_heads, tokens = table_width * page;
  const Plans p = plans_of(seqs, max_q, n_groups, max_group, max_prefix, max_tail, ratio, kv_heads, head_dim, group,
                           tokens, T);
  if (!workspace || workspace_bytes < bytes_of(p, T, q_heads, head_dim)) return QMM_EWORKSPACE;
  if (!aligned(workspace, 16)) return QMM_EALIGN;
  // (a launch holds 2^32 threads; those for many rows have up to 512 a block)
  if (p.prefix.blocks >= int64_t{1} << (p.prefix.ws ? 24 : 23) || p.prefix.blocks + p.own.blocks >= (int64_t{1} << 24))
    return QMM_ERANGE;
  SharedArgs a{};
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
  a.scale_log2 = scale * 1.44269504088896341f;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.splits = static_cast<int32_t>(p.own.splits);
  a.row_tiles = static_cast<int32_t>(p.own.row_tiles);
  a.least = a.p_least = static_cast<int32_t>(kLeastSteps);
  a.round = static_cast<int32_t>(p.round);
  a.groups = groups;
  a.prefix = prefix;
  a.n_groups = static_cast<int32_t>(n_groups);
  a.p_splits = static_cast<int32_t>(p.prefix.splits);
  a.p_row_tiles = static_cast<int32_t>(p.prefix.row_tiles);
  a.p_round = static_cast<int32_t>(p.p_round);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + T * q_heads * (p.prefix.splits + p.own.splits) * head_dim);
  if (dtype == QMM_BF16) prefix_attention_bf16(a, p.prefix, p.own, p.together, as_stream(stream));
  else prefix_attention_f16(a, p.prefix, p.own, p.together, as_stream(stream));
  return launch_status();
}
