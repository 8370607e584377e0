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

}  // namespace qmm
