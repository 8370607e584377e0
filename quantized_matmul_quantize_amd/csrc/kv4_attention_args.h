// kv4_attention_args.h -- arguments and launch plan of the attention kernels.
#pragma once

#include "kv4_device.h"

namespace qmm {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kStep = 32;            // keys per step: one k-extent of the second product
constexpr int kBeyond = 1 << 30;     // a key no context reaches

struct AttnArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const int32_t* cu_q;
  const int32_t* context;
  const int32_t* table;
  int64_t table_stride;
  const uint8_t* cache;
  Kv4Shape sh;
  int32_t T, q_heads, ratio, seqs;
  int32_t limit;                     // tokens the table holds
  int32_t window, sinks;             // window 0: none
  float scale_log2;                  // scale * log2(e)
  uint16_t* out;
  float* lse;
  // work split: `splits` chunks of `chunk` steps, `row_tiles` blocks over the rows of a sequence
  int32_t splits, chunk, row_tiles;
  float* part_o;                     // [T * q_heads][splits][D]
  float2* part_ml;                   // [T * q_heads][splits]
};

// The same for a batch in groups that share a prefix (kv4_prefix.hip).  A
// group's prefix is one work item, whose rows are the queries of all of its
// sequences and see every key; each sequence's own keys are another.
struct SharedArgs : AttnArgs {
  const int32_t* groups;             // [n_groups + 1] first sequences
  const int32_t* prefix;             // [n_groups] tokens
  int32_t n_groups;
  // The prefixes' split: chunks at most, their steps at least and in multiples
  // of, blocks over the rows; a sequence's own: as before, `splits` chunks at most.
  int32_t p_splits, p_least, p_round, p_row_tiles;
  int32_t least, round;
};
// Whose keys a block takes: those of a sequence, of a group's prefix, or a
// sequence's own behind it.
enum Part { kWhole, kPrefix, kOwn };

// A sequence's queries: rows of q, and the position of the first.
struct Sequence {
  int row0, n, first, ctx;
};
__device__ __forceinline__ Sequence sequence_of(const AttnArgs& a, int b) {
  Sequence s;
  int r0 = b, r1 = b + 1;
  if (a.cu_q) {
    r0 = min(max(a.cu_q[b], 0), a.T);
    r1 = min(max(a.cu_q[b + 1], r0), a.T);
  }
  s.row0 = r0;
  s.n = r1 - r0;
  s.ctx = min(max(a.context[b], 0), a.limit);
  s.first = s.ctx - s.n;
  return s;
}

// The steps of keys that queries first .. last (positions) need: `sink_steps`
// from key 0, then from key `start`, `count` in all.
struct Steps {
  int sink_steps, start, count;
  __device__ __forceinline__ int key(int s) const { return s < sink_steps ? s * kStep : start + (s - sink_steps) * kStep; }
};
__device__ __forceinline__ Steps steps_of(const AttnArgs& a, int first, int last) {
  Steps s{0, 0, 0};
  if (last < 0) return s;
  if (a.window > 0) {
    const int low = max(0, first - a.window + 1) & ~(kStep - 1);
    s.sink_steps = min((min(a.sinks, low) + kStep - 1) / kStep, low / kStep);
    s.start = low;
  }
  s.count = s.sink_steps + (last - s.start) / kStep + 1;
  return s;
}

// ---- parts of a batch with shared prefixes.  Keys of a prefix are counted in
// whole steps: the others of its last one are taken with each sequence's own.
__device__ __forceinline__ int prefix_keys(const SharedArgs& a, int g) {
  return min(max(a.prefix[g], 0), a.limit) & ~(kStep - 1);
}
// Whether every query of a sequence sees all of a prefix's keys.  One that does
// not is attended to by itself.
__device__ __forceinline__ bool shares(const Sequence& s, int keys) { return keys > 0 && s.n > 0 && s.first + 1 >= keys; }

// `count` steps in at most `splits` chunks of whole rounds, none below `least`.
struct Chunks {
  int chunk, chunks;
};
__device__ __forceinline__ int steps_in(int keys) { return (max(keys, 0) + kStep - 1) / kStep; }
__device__ __forceinline__ Chunks chunks_of(int count, int splits, int least, int round) {
  const int even = (count + splits - 1) / splits;
  const int chunk = (max(max(even, least), 1) + round - 1) / round * round;
  return {chunk, max(1, (count + chunk - 1) / chunk)};
}

struct Item {
  Sequence sq;
  int table_row;
  int lo;            // its first key
  bool shared;       // its rows have a prefix's part too
};
// The group of a sequence, -1 for none.  All lanes of the wavefront.
__device__ __forceinline__ int group_of(const SharedArgs& a, int b) {
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;
  for (int i = 0; i <= a.n_groups; i += kWave) {
    const bool starts = i + lane <= a.n_groups && a.groups[i + lane] <= b;
    before += __popcll(__ballot(starts));
  }
  return before - 1 < a.n_groups ? before - 1 : -1;
}
__device__ __forceinline__ Item own_item(const SharedArgs& a, int b) {
  Item x{sequence_of(a, b), b, 0, false};
  const int g = __builtin_amdgcn_readfirstlane(group_of(a, b));
  const int keys = g < 0 ? 0 : prefix_keys(a, g);
  x.shared = shares(x.sq, keys);
  x.lo = x.shared ? keys : 0;
  return x;
}
// A group's prefix: rows of all of its sequences; read through the pages of the
// first that shares it (no keys where none does).
__device__ __forceinline__ Item prefix_item(const SharedArgs& a, int g) {
  const int lane = threadIdx.x & (kWave - 1);
  const int s0 = min(max(a.groups[g], 0), a.seqs), s1 = min(max(a.groups[g + 1], s0), a.seqs);
  const int keys = prefix_keys(a, g);
  int leader = -1;
  for (int i = s0; i < s1 && leader < 0; i += kWave) {
    const bool one = i + lane < s1 && shares(sequence_of(a, min(i + lane, s1 - 1)), keys);
    const uint64_t who = __ballot(one);
    if (who) leader = i + __builtin_ctzll(who);
  }
  Item x{};
  x.table_row = __builtin_amdgcn_readfirstlane(max(leader, 0));
  x.shared = true;
  int r0 = s0, r1 = s1;
  if (a.cu_q) {
    r0 = min(max(a.cu_q[s0], 0), a.T);
    r1 = min(max(a.cu_q[s1], r0), a.T);
  }
  x.sq.row0 = r0;
  x.sq.n = r1 - r0;
  x.sq.ctx = leader < 0 ? 0 : keys;
  x.sq.first = x.sq.ctx;
  return x;
}
__device__ __forceinline__ Item item_of(const AttnArgs& a, int b) { return {sequence_of(a, b), b, 0, false}; }
template <Part PART>
__device__ __forceinline__ Chunks part_chunks(const SharedArgs& a, const Item& x) {
  const int count = steps_in(x.sq.ctx - x.lo);
  if constexpr (PART == kPrefix) return chunks_of(count, a.p_splits, a.p_least, a.p_round);
  else return chunks_of(count, a.splits, a.least, a.round);
}
template <Part PART>
__device__ __forceinline__ Item item_of(const SharedArgs& a, int b) {
  if constexpr (PART == kPrefix) return prefix_item(a, b);
  else return own_item(a, b);
}

// Column tiles of 16 rows a wavefront takes of more than 16 rows (in a chunk
// kernel, of a chunk's), and whether it can take two steps at once of few: by
// the registers that the sums (D / 16 a tile) and a group's products, scales
// and zero-points need.  Two tiles halve what a product reads of LDS: three
// chunks of prompts, D 128 in one group, 830 us against 1270; but in two groups
// they no longer fit, 470 us against 215 for 2 x 1024 queries at 6000 keys.
constexpr int attention_tiles(int D, int group) { return D < 256 && D / group < 4 ? 2 : 1; }
constexpr int attention_chunk_tiles(int D, int group) { return D * (D / group) <= 128 ? 2 : 1; }
constexpr bool attention_pairs(int D, int group) { return D < 256 || group > 32; }

struct AttnPlan {
  int pk, nt;         // steps a wavefront takes at once, column tiles
  bool ws;            // wavefronts of a block share the rows and split the keys
  int64_t rows;       // rows of a block
  int64_t row_tiles, splits, chunk, max_q, blocks;
};

void attention_bf16(const AttnArgs& a, const AttnPlan& p, hipStream_t s);
void attention_f16(const AttnArgs& a, const AttnPlan& p, hipStream_t s);

// (together: both parts in one launch, by the prefix's kernel)
void prefix_attention_bf16(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s);
void prefix_attention_f16(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s);

}  // namespace qmm
