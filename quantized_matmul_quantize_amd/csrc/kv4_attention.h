// kv4_attention.h -- the kernels of kv4_attention.hip (causal attention over
// the 4-bit paged cache; the format and the masks are stated in
// include/qmm.h), instantiated for one type of q per source file.
//
// The rows of one sequence and kv head (its queries times the query heads that
// share the kv head) stand in the 16 columns of the products, the keys are
// taken 32 at a time (a step), in one pass with a running maximum and sum:
//
//   S^T = K Q^T   codes of 16 keys x 32 channels as the first operand, q as the
//                 second, so a lane ends with 4 keys of one column;
//   O^T += V^T P^T  codes of 16 channels x 32 keys first, the same lane's
//                 probabilities second: the lane that computed S^T[4 kb + i][r]
//                 of two 16-key tiles holds exactly the eight k-entries that
//                 the second product wants of it, so the probabilities never
//                 leave their lane, and the running statistics of column r
//                 belong to the lanes that hold column r of O^T.
//
// The codes enter the matrix cores as they are, as the binary16 numbers
// off + c, exactly; offset, zero-point and scale are applied around the products:
//   x[t] = sum_g s[t,g] ((sum_{d in g} q_d (16 + c)) - (16 + z[t,g]) sum_{d in g} q_d)
//   o[d] = 2^e[g] (sum_t p'[t] (64 + c) - sum_t p'[t] (64 + z[t,g])),  p' = p s[t,g] 2^-e[g]
// with the second sum of o one more product whose first operand is 64 + z.  (An
// offset of 64 takes one shift a word less than 16, but its rounding is the
// scores' largest error; bf16 operands would need 128.)  bf16 queries are first
// scaled by a power of two, their largest to 2^14 .. 2^15: exact but for what
// lies 2^31 below it.  p' is rounded to binary16 (2^-11) for either type of q:
// bf16 would cost 2^-8.  Its range is kept by two powers of two of each row, of
// the keys that it sees, that are moved only when they must be: p lies below
// 2^15 (and reaches 2^7 where the maximum was last moved, so that what is lost
// below 2^-25 is 2^-32 of the largest), s 2^-e below 1.  The scores, maxima and
// sums of p stay in fp32.
//
// What bounds decode is the vector unit, not the matrix cores: two operations
// a pair of codes to make operands of them, and then the arithmetic on the
// scores, of which few rows leave most columns idle.  So with few rows a
// wavefront takes two steps at once (PK = 2): both halves of the columns
// hold the same rows but keep the scores, maxima, sums and results of a step
// of their own, and are joined at the end, as the wavefronts are.  (Four steps
// at once for 4 rows: 220 instead of 250 vector operations a step, but 70 KiB
// of LDS a block and 58 instead of 54 us for 64 sequences of 4096 tokens.)
// These take 53 us (8 kv heads of 128 in one group, 243 MB: 4.6 TB/s), of which
// loads alone are 45, the arithmetic alone (before the row's own powers of two)
// 44; 2 sequences of 131072 tokens in groups of 64 (293 MB) 65, of which 52, 51.
#pragma once

#include "kv4_attention_args.h"

namespace qmm {
namespace {

// Eight codes of a word as four pairs 64 + c: bits 4-7 of 0x5400 (64.0) are
// worth 1, so one of the pairs needs no shift.  (16 + c, nibbles at bits 6-9:
// Int4Magic<QMM_F16>.)
struct Codes64 {
  static constexpr uint32_t magic = 0x54005400u;
  static constexpr uint32_t mask = 0x00F000F0u;
  template <int N>
  static __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t m) {
    return ((N == 0 ? w << 4 : w >> (N == 0 ? 0 : 4 * N - 4)) & mask) | m;
  }
  static __device__ __forceinline__ void unpack(uint32_t w, uint32_t m, uint32_t p[4]) {
    p[0] = pair<0>(w, m);
    p[1] = pair<1>(w, m);
    p[2] = pair<2>(w, m);
    p[3] = pair<3>(w, m);
  }
};

// Queries as second operands.  The power of two that takes the largest finite
// one to 2^14 .. 2^15 (held to normal numbers), and its inverse.
struct QueryScale {
  float down, up;
};
template <int N>
__device__ __forceinline__ float largest_bf16(const u32x4 (&q)[N], float most) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float a = fabsf(bf16lo_to_f32(q[j][w])), b = fabsf(bf16hi_to_f32(q[j][w]));
      most = fmaxf(most, a < INFINITY ? a : 0.0f);    // infinities and NaN are their own row's
      most = fmaxf(most, b < INFINITY ? b : 0.0f);
    }
  return most;
}
__device__ __forceinline__ QueryScale query_scale(float most) {
  const int e = min(max(static_cast<int>(__float_as_uint(most) >> 23), 27), 254);
  return {__uint_as_float(static_cast<uint32_t>(268 - e) << 23), __uint_as_float(static_cast<uint32_t>(e - 14) << 23)};
}
template <int N>
__device__ __forceinline__ void to_f16(u32x4 (&q)[N], float down) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int w = 0; w < 4; ++w)
      q[j][w] = pack_pair<QMM_F16>(bf16lo_to_f32(q[j][w]) * down, bf16hi_to_f32(q[j][w]) * down);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0,
                                                0);
}
// p s of a pair of keys, each rounded once
__device__ __forceinline__ uint32_t weighted(float p0, float p1, f16x2_t s) {
  const f16x2_t w{static_cast<_Float16>(p0 * static_cast<float>(s[0])),
                  static_cast<_Float16>(p1 * static_cast<float>(s[1]))};
  return __builtin_bit_cast(uint32_t, w);
}

__device__ __forceinline__ float max_over_quads(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum_over_quads(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}
__device__ __forceinline__ f16x2_t pk_max(f16x2_t a, f16x2_t b) { return __builtin_elementwise_max(a, b); }
__device__ __forceinline__ f16x2_t pair16(float v) {
  return f16x2_t{static_cast<_Float16>(v), static_cast<_Float16>(v)};
}
// Powers of two for values of the scales that a row sees and of those it does
// not: the row's own largest goes to 2^-3 .. 2^-2, and no other may pass 2^14,
// as its probability of 0 would meet an infinity.  (A scale is below 2^16.)
__device__ __forceinline__ float shrink_for(float largest) {
  return __uint_as_float((251u - (__float_as_uint(largest) >> 23)) << 23);
}
__device__ __forceinline__ float shrink_for_hidden(float largest) {
  return __uint_as_float(min(267u - (__float_as_uint(largest) >> 23), 254u) << 23);
}
__device__ __forceinline__ float larger(f16x2_t v) { return fmaxf(static_cast<float>(v[0]), static_cast<float>(v[1])); }
__device__ __forceinline__ bool past_one(f16x2_t v) {
  return v[0] > static_cast<_Float16>(1.0f) || v[1] > static_cast<_Float16>(1.0f);
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// What a base that moves from `from` to `to` for scores up to `top` (less `from`)
// leaves of them but 7, where that is more than 1.  Past 2^24 the base's rounding
// does, past 2^31 by more than an exponential has room for: scores are then taken
// less this too.  (So large they are known no better than that.)
__device__ __forceinline__ float unrounded(float top, float from, float to, bool moved) {
  const float rest = top + (from - to) - 7.0f;
  return rest > 1.0f || (rest < -1.0f && moved) ? rest : 0.0f;
}
// log sum exp from the base-2 maximum and the sum, and what results are divided
// by.  A sum of 0 is that of no key; one that is not a number is its row's.
__device__ __forceinline__ float lse_of(float base, float sum) {
  return sum == 0.0f ? -INFINITY : (base + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f;
}
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }
// A part's sum at the maximum of all parts: one without a maximum saw no key or
// none that is a number, and adds what it has.
__device__ __forceinline__ float sum_at(float sum, float m, float most) {
  return m == -INFINITY ? sum : sum * exp2_fast(m - most);
}

// Shape of the kernel for few rows: PK as above, NT column tiles.  The
// wavefronts of a block share the rows and take every fourth unit of PK steps
// each.  (Many rows: kv4_attention_chunk.h.)
template <int D, int GROUP, int PK, int NT>
struct Shape {
  static constexpr int kG = D / GROUP;
  static constexpr int kCols = 16 / PK;                     // rows in 16 columns
  static constexpr int kRows = kCols * NT;
  static constexpr int kMTiles = GROUP / 16;                // channel tiles of a group
  static constexpr int kSteps = D / 32;                     // k-extents of a key
  static constexpr int kChunks = D / 32;                    // 16-byte pieces of a key's codes
  // A unit's keys and values have LDS slots of their own: the keys of the next
  // unit are requested as soon as this one's scores are taken, its values
  // after the sums, so half a unit or more is always on its way.  Units of one
  // step have two slots each.
  static constexpr int kSlots = PK == 1 ? 2 : 1;
  static constexpr int kKTile = 8 * D + 128 * kG;           // 16 keys: codes, then K and V params [g][16]
  static constexpr int kVTile = 8 * D;
  static constexpr int kKSlot = PK * 2 * kKTile, kVSlot = PK * 2 * kVTile;
  static constexpr int kWaveBytes = kSlots * (kKSlot + kVSlot);
  // loads of a 16-key tile: 1 KiB each, for D = 64 codes and params in one
  static constexpr int kCodeLoads = D / 128;
  static constexpr int kKLoads = PK * 2 * (D == 64 ? 1 : kCodeLoads + 1);
  static constexpr int kVLoads = PK * 2 * (D == 64 ? 1 : kCodeLoads);
  // the epilogue's sums: 16 columns of D channels a wavefront
  static constexpr int kPad = D + 4;
  static_assert(kWaveBytes >= (16 * kPad + 32) * 4, "the epilogue reuses the slots");
  // Rotation of a key's pieces within its row in LDS: the 16 lanes that read
  // one piece of 16 keys then meet every bank once.
  static __device__ __forceinline__ int rot(int r) { return r * kChunks / 16; }
};

// Where a part's results go: chunk `split` of a row's slots in the workspace.
template <Part PART, typename A>
__device__ __forceinline__ int64_t slot_of(const A& a, int64_t rh, int split) {
  if constexpr (PART == kWhole) return rh * a.splits + split;
  else return rh * (a.p_splits + a.splits) + (PART == kPrefix ? 0 : a.p_splits) + split;
}

template <int DT, int D, int GROUP, int PK, int NT, Part PART, typename A>
__device__ __forceinline__ void attention_block(const A& a, uint32_t id, uint8_t* lds) {
  static_assert(PK == 1 || NT == 1, "steps are taken together for few rows only");
  using L = Shape<D, GROUP, PK, NT>;
  constexpr int G = L::kG, MT = L::kMTiles, kSteps = L::kSteps;
  constexpr float kOff = Int4Magic<QMM_F16>::offset;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r = lane & 15, kb = lane >> 4;
  const int bank = PK == 1 ? 0 : r / L::kCols;              // the step of a unit that column r keeps

  int32_t splits = a.splits, row_tiles = a.row_tiles;
  if constexpr (PART == kPrefix) {
    splits = a.p_splits;
    row_tiles = a.p_row_tiles;
  }
  const int split = static_cast<int>(id % splits);
  id /= splits;
  const int kvh = static_cast<int>(id % a.sh.heads);
  id /= a.sh.heads;
  const int tile0 = static_cast<int>(id % row_tiles);
  const int b = static_cast<int>(id / row_tiles);
  Item item;
  if constexpr (PART == kWhole) item = item_of(a, b);
  else item = item_of<PART>(a, b);
  const Sequence sq = item.sq;
  const int rows = sq.n * a.ratio;

  // Byte offsets of this lane's loads in a record: at + place * per.
  int k_at[D == 64 ? 1 : L::kCodeLoads], v_at[D == 64 ? 1 : L::kCodeLoads];
  int k_per = D / 2;
  int p_at = a.sh.page * D + (lane / 4) * a.sh.page * 4 + 16 * (lane & 3);   // [K, V][group][page] words
#pragma unroll
  for (int n = 0; n < (D == 64 ? 1 : L::kCodeLoads); ++n) {
    const int p = 64 * n + lane, R = p / L::kChunks;
    k_at[n] = R * (D / 2) + 16 * ((p - L::rot(R)) & (L::kChunks - 1));
    v_at[n] = a.sh.page * (D / 2) + 16 * p;
  }
  if (D == 64 && lane >= 32) {
    const int q = lane - 32;
    k_at[0] = a.sh.page * D + (q / 4) * a.sh.page * 4 + 16 * (q & 3);
    k_per = 4;
  }
  const int record = static_cast<int>(a.sh.record_bytes());
  const uint32_t page_bytes = static_cast<uint32_t>(a.sh.heads) * static_cast<uint32_t>(record);
  const uint8_t* head = a.cache + static_cast<int64_t>(kvh) * record;
  uint8_t* const mine = lds + wave * L::kWaveBytes;
  const uint32_t mine_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(mine));
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const table_t table = (table_t)(a.table + item.table_row * a.table_stride);

  // A 16-key tile past the context, or whose page is not of this cache, is
  // read through an empty resource: zeros, so scales of 0.
  const uint32_t pages = static_cast<uint32_t>(a.sh.pages);
  auto tile_of = [&](int page) {
    const bool here = static_cast<uint32_t>(page) < pages;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(head + static_cast<uint64_t>(static_cast<uint32_t>(here ? page : 0)) * page_bytes), 0,
        here ? record : 0, kBufferWord3);
  };
  struct Unit {           // the steps of a unit: their first keys and the pages of their 16-key tiles
    int key[PK], page[2 * PK];
  };

  for (int tile = tile0; tile * L::kRows < rows; tile += row_tiles) {
    const int row_lo = tile * L::kRows;
    const int row_hi = min(row_lo + L::kCols * NT, rows) - 1;
    // (rows of a prefix see all of its keys)
    const int pos_lo = PART == kPrefix ? kBeyond - 1 : sq.first + row_lo / a.ratio;
    const int pos_hi = row_hi < row_lo ? -1 : sq.first + row_hi / a.ratio;
    Steps st;
    Chunks ch;
    if constexpr (PART == kWhole) {
      st = steps_of(a, sq.first + tile * L::kRows / a.ratio,
                    sq.first + (min((tile + 1) * L::kRows, rows) - 1) / a.ratio);
      ch = {a.chunk, max(1, (st.count + a.chunk - 1) / a.chunk)};
    } else {
      // (chunks by all of the part's keys, as they are joined; a sequence's own up to what the tile's last row sees)
      const int end = PART == kPrefix ? sq.ctx : min(sq.ctx, sq.first + (min((tile + 1) * L::kRows, rows) - 1) / a.ratio + 1);
      st = {0, item.lo, steps_in(end - item.lo)};
      ch = part_chunks<PART>(a, item);
    }
    const int chunk = ch.chunk, chunks = ch.chunks;
    if (split >= chunks) continue;
    const int s_lo = split * chunk + wave * PK, s_hi = min(split * chunk + chunk, st.count);
    constexpr int kStride = PK * kWaves;

    auto unit_of = [&](int s) {
      Unit x;
#pragma unroll
      for (int c = 0; c < PK; ++c) {
        x.key[c] = s + c < s_hi ? st.key(s + c) : kBeyond;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = x.key[c] + 16 * u;
          const int page = table[max(min(t, sq.ctx - 1), 0) >> a.sh.shift];
          x.page[2 * c + u] = t < sq.ctx ? page : -1;
        }
      }
      return x;
    };
    auto issue_keys = [&](const Unit& x, int slot) {
      const uint32_t dst = mine_at + slot * L::kKSlot;
#pragma unroll
      for (int i = 0; i < 2 * PK; ++i) {
        const __amdgpu_buffer_rsrc_t rs = tile_of(x.page[i]);
        const int place = (x.key[i / 2] + 16 * (i % 2)) & (a.sh.page - 1);
        if constexpr (D == 64) {
          if (lane < 32 + 8 * G)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(dst + i * L::kKTile), 16,
                                                     k_at[0] + place * k_per, 0, 0, 0);
        } else {
#pragma unroll
          for (int n = 0; n < L::kCodeLoads; ++n)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(dst + i * L::kKTile + n * 1024), 16,
                                                     k_at[n], place * (D / 2), 0, 0);
        }
      }
      if (D != 64 && lane < 8 * G) {
#pragma unroll
        for (int i = 0; i < 2 * PK; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(tile_of(x.page[i]),
                                                   (lds_ptr_t)(uintptr_t)(dst + i * L::kKTile + 8 * D), 16, p_at,
                                                   ((x.key[i / 2] + 16 * (i % 2)) & (a.sh.page - 1)) * 4, 0, 0);
      }
    };
    auto issue_values = [&](const Unit& x, int slot) {
#pragma unroll
      for (int c = 0; c < PK; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const __amdgpu_buffer_rsrc_t rs = tile_of(x.page[2 * c + u]);
          const int place = (x.key[c] + 16 * u) & (a.sh.page - 1);
          const uint32_t dst = mine_at + L::kSlots * L::kKSlot + slot * L::kVSlot + (2 * c + u) * L::kVTile;
#pragma unroll
          for (int n = 0; n < (D == 64 ? 1 : L::kCodeLoads); ++n)
            if (D != 64 || lane < 32)
              __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(dst + n * 1024), 16, v_at[n],
                                                       place * (D / 2), 0, 0);
        }
    };

    // the first units are on their way while q is read
    Unit now = unit_of(s_lo), next = unit_of(s_lo + kStride);
    if (s_lo < s_hi) {
      issue_keys(now, 0);
      issue_values(now, 0);
      if (L::kSlots == 2) {
        issue_keys(next, 1);
        issue_values(next, 1);
      }
    }

    // queries as second operands, their sums per group, and their positions
    u32x4 qv[NT][kSteps];
    float qsum[NT][G];
    int pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row_lo + 16 * n + r % L::kCols;
      const bool live = row < rows;
      const int tok = live ? row / a.ratio : 0, qh = live ? kvh * a.ratio + row - tok * a.ratio : 0;
      pos[n] = !live ? -1 : PART == kPrefix ? kBeyond - 1 : sq.first + tok;
      const uint16_t* qp = a.q + (sq.row0 + tok) * a.q_ts + qh * a.q_hs + 8 * kb;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) qv[n][j] = live ? ld16(qp + 32 * j) : u32x4{0u, 0u, 0u, 0u};
    }
    // (the power of two of bf16 queries is that of all rows, which are a sequence's;
    // in a prefix each row's own: no sequence's queries cost another's bits)
    constexpr bool kApart = PART == kPrefix;
    float key_scale[kApart ? NT : 1];
#pragma unroll
    for (int n = 0; n < (kApart ? NT : 1); ++n) key_scale[n] = a.scale_log2;
    if constexpr (DT == QMM_BF16 && kApart) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const QueryScale qs = query_scale(max_over_quads(largest_bf16(qv[n], 0.0f)));
        key_scale[n] *= qs.up;
        to_f16(qv[n], qs.down);
      }
    } else if constexpr (DT == QMM_BF16) {
      float most = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) most = largest_bf16(qv[n], most);
      const QueryScale qs = query_scale(wave_max(most));
      key_scale[0] *= qs.up;
#pragma unroll
      for (int n = 0; n < NT; ++n) to_f16(qv[n], qs.down);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float s = 0.0f;
#pragma unroll
        for (int j = g * GROUP / 32; j < (g + 1) * GROUP / 32; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w) s += f16lo_to_f32(qv[n][j][w]) + f16hi_to_f32(qv[n][j][w]);
        qsum[n][g] = sum_over_quads(s);
      }

    f32x4 o[NT][G][MT], corr[NT][G];
    // p = 2^(x - base); base is -inf until a key is seen, then at least 2^-15
    // below and at most 2^7 above the largest x
    float base[NT], l[NT];
    f16x2_t shrink[NT][G];  // 2^-e[g], the column's, twice
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      base[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        shrink[n][g] = pair16(32768.0f);
        corr[n][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < MT; ++x) o[n][g][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    const uint32_t magic_q = vgpr_const(Int4Magic<QMM_F16>::kMagic);
    const uint32_t magic_v = vgpr_const(Codes64::magic);

    float p[NT][8];                // probabilities of a unit, and the pairs of scales and zero-points of its values
    uint32_t sv[G][4], zv[G][4];

    auto scores = [&](int s, const Unit& unit, int slot_n) {
      const uint8_t* slot = mine + slot_n * L::kKSlot;
      // ---- products, a unit's step kept in its own columns
      f32x4 prod[NT][G][2];
#pragma unroll
      for (int c = 0; c < PK; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* kp = slot + (2 * c + u) * L::kKTile;
          uint32_t w[kSteps];
          if constexpr (D == 64) {
            const u32x2 v =
                *reinterpret_cast<const u32x2*>(kp + 16 * (2 * r + (((kb >> 1) + L::rot(r)) & 1)) + 8 * (kb & 1));
            w[0] = v.x;
            w[1] = v.y;
          } else {
#pragma unroll
            for (int h = 0; h < D / 128; ++h) {
              const int piece = (D / 128) * kb + h;
              const u32x4 v = *reinterpret_cast<const u32x4*>(
                  kp + 16 * (L::kChunks * r + ((piece + L::rot(r)) & (L::kChunks - 1))));
#pragma unroll
              for (int j = 0; j < 4; ++j) w[4 * h + j] = v[j];
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            f32x4 acc[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float i = -kOff * qsum[n][g];
              acc[n] = f32x4{i, i, i, i};
            }
#pragma unroll
            for (int j = g * GROUP / 32; j < (g + 1) * GROUP / 32; ++j) {
              uint32_t av[4];
              Int4Magic<QMM_F16>::unpack(w[j], magic_q, av);
#pragma unroll
              for (int n = 0; n < NT; ++n) acc[n] = mfma(u32x4{av[0], av[1], av[2], av[3]}, qv[n][j], acc[n]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) prod[n][g][u][i] = c == 0 || bank == c ? acc[n][i] : prod[n][g][u][i];
          }
        }
      // ---- what this lane's keys are: 4 of each 16-key tile of its step
      int t0 = unit.key[0];
#pragma unroll
      for (int c = 1; c < PK; ++c) t0 = bank == c ? unit.key[c] : t0;
      int holes = 0;
#pragma unroll
      for (int i = 0; i < 2 * PK; ++i) holes |= static_cast<uint32_t>(unit.page[i]) < pages ? 0 : 1 << i;
      const int first = unit.key[0], end = unit.key[PK - 1] + kStep;
      const bool whole = holes == 0 && end - first == PK * kStep && end - 1 <= pos_lo &&
                         (a.window == 0 || first > pos_hi - a.window || end <= a.sinks);
      const int mine_missing = holes >> (2 * bank);
      // ---- scores
      const uint8_t* params = slot + 2 * bank * L::kKTile + 8 * D + 16 * kb;
      f32x4 x[NT][2];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 par = *reinterpret_cast<const u32x4*>(params + u * L::kKTile + g * 64);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float ks = kv4_scale(par[i]), z = kv4_zero(par[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float sc = ks * key_scale[kApart ? n : 0];
              const float v = fmaf(-z, qsum[n][g], prod[n][g][u][i]);
              x[n][u][i] = g == 0 ? sc * v : fmaf(sc, v, x[n][u][i]);
            }
          }
        }
      // The memory of a hidden key may hold anything: its scores are replaced
      // whatever they are, and its values' scale is taken as 0 where no row of
      // the lane sees it (0 times a NaN would be one).  Codes and zero-points
      // are finite whatever their bits.
      uint32_t keep[NT][4];          // bits of the pairs of scales that a row sees
      if (!whole) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) keep[n][e] = 0u;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 16 * u + 4 * kb + i;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const bool seen = !((mine_missing >> u) & 1) && t <= pos[n] &&
                                (a.window == 0 || t > pos[n] - a.window || t < a.sinks);
              x[n][u][i] = seen ? x[n][u][i] : -INFINITY;
              keep[n][2 * u + i / 2] |= seen ? 0xFFFFu << (16 * (i & 1)) : 0u;
            }
          }
      }
      // ---- scales of the values, pairs of keys; the running powers of two, by
      // the scales that a row sees: a key that is hidden from it, such as a later
      // token, must not cost it bits
      f16x2_t most[G];
      bool grow = false;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x4 par[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          par[u] = *reinterpret_cast<const u32x4*>(params + u * L::kKTile + G * 64 + g * 64);
        most[g] = f16x2_t{0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t p0 = par[e >> 1][2 * (e & 1)], p1 = par[e >> 1][2 * (e & 1) + 1];
          zv[g][e] = (__builtin_amdgcn_perm(p1, p0, 0x0c060c02u) << 4) | magic_v;
          sv[g][e] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
          if (!whole) sv[g][e] &= NT == 1 ? keep[0][e] : keep[0][e] | keep[NT - 1][e];
          most[g] = pk_max(most[g], __builtin_bit_cast(f16x2_t, sv[g][e]));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) grow |= past_one(most[g] * shrink[n][g]);
      }
      // ---- running maximum and powers of two: one test for both
      float top[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float t = max3(x[n][0][0], x[n][0][1], x[n][0][2]);
        t = max3(t, x[n][0][3], x[n][1][0]);
        t = max3(t, x[n][1][1], x[n][1][2]);
        t = max3(t, x[n][1][3], x[n][1][3]);
        top[n] = t;
        grow |= t > base[n] + 15.0f;
      }
      if (__any(grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // 2^7 at the new maximum; columns that have seen no key stay at -inf
          const float to = fmaxf(base[n], max_over_quads(top[n]) - 7.0f);
          const float fade = to == -INFINITY ? 1.0f : exp2_fast(base[n] - to);
          base[n] = to;
          l[n] *= fade;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            f16x2_t own = most[g];
            if (NT > 1 && !whole) {
              own = f16x2_t{0, 0};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t seen = sv[g][e] & keep[n][e];
                own = pk_max(own, __builtin_bit_cast(f16x2_t, seen));
              }
            }
            const float now_shrink = static_cast<float>(shrink[n][g][0]);
            float next_shrink = fminf(now_shrink, shrink_for(max_over_quads(larger(own))));
            if (NT > 1) next_shrink = fminf(next_shrink, shrink_for_hidden(max_over_quads(larger(most[g]))));
            const float f = fade * (next_shrink / now_shrink);
            shrink[n][g] = pair16(next_shrink);
            corr[n][g] *= f;
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= f;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float from = base[n] == -INFINITY ? 0.0f : base[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[n][2 * e] = exp2_fast(x[n][e >> 1][2 * (e & 1)] - from);
          p[n][2 * e + 1] = exp2_fast(x[n][e >> 1][2 * (e & 1) + 1] - from);
          l[n] += p[n][2 * e] + p[n][2 * e + 1];
        }
      }
    };

    auto sums = [&](int slot_n) {
      const uint8_t* slot = mine + L::kSlots * L::kKSlot + slot_n * L::kVSlot;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x4 pv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pv[n][e] = weighted(p[n][2 * e], p[n][2 * e + 1],
                                __builtin_bit_cast(f16x2_t, sv[g][e]) * shrink[n][g]);
          // row m of the first operand holds the zero-points of m's own step,
          // so column r finds its sum where 4 kb + i belongs to r's step
          corr[n][g] = mfma(u32x4{zv[g][0], zv[g][1], zv[g][2], zv[g][3]}, pv[n], corr[n][g]);
        }
#pragma unroll
        for (int c = 0; c < PK; ++c) {
          u32x4 vw[2], pc[NT];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            vw[u] = *reinterpret_cast<const u32x4*>(slot + (2 * c + u) * L::kVTile + kb * 2 * D +
                                                    16 * (g * (GROUP / 8) + (r & (GROUP / 8 - 1))));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) pc[n][e] = PK == 1 || bank == c ? pv[n][e] : 0u;
          // key pairs of this lane's word, word half or word byte (16, 8 or 4 words a group)
          constexpr int kParts = GROUP == 128 ? 2 : 1;
#pragma unroll
          for (int part = 0; part < kParts; ++part) {
            uint32_t unit[4];
            uint32_t sel;
            if constexpr (GROUP == 128) sel = part ? 0x07060302u : 0x05040100u;
            else if constexpr (GROUP == 64) sel = (r >> 3) ? 0x07060302u : 0x05040100u;
            else sel = 0x0c040c00u + (r >> 2) * 0x00010001u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              unit[e] = __builtin_amdgcn_perm(vw[e >> 1][2 * (e & 1) + 1], vw[e >> 1][2 * (e & 1)], sel);
#pragma unroll
            for (int y = 0; y < MT / kParts; ++y) {
              u32x4 av;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                av[e] = ((y == 0 ? unit[e] << 4 : unit[e] >> (4 * y - 4)) & Codes64::mask) | magic_v;
#pragma unroll
              for (int n = 0; n < NT; ++n)
                o[n][g][part * (MT / kParts) + y] = mfma(av, pc[n], o[n][g][part * (MT / kParts) + y]);
            }
          }
        }
      }
    };

    int slot = 0;
    for (int s = s_lo; s < s_hi; s += kStride) {
      const bool more = s + L::kSlots * kStride < s_hi;       // the unit requested in this round exists
      const bool last = s + kStride >= s_hi;
      // with two slots `after` follows `next`
      Unit after = L::kSlots == 2 ? unit_of(s + 2 * kStride) : next;
      __builtin_amdgcn_sched_barrier(0);
      // this unit's keys: behind them only its values and the other slot's unit
      if (L::kSlots == 2 && !last) wait_vm<L::kKLoads + 2 * L::kVLoads>();
      else wait_vm<L::kVLoads>();
      asm volatile("" ::: "memory");
      scores(s, now, slot);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);                     // LDS reads done: the slot may be requested again
      __builtin_amdgcn_sched_barrier(0);
      if (more) issue_keys(after, slot);
      // this unit's values: behind them the other slot's unit and the keys just requested
      if (L::kSlots == 2) {
        if (more) wait_vm<2 * L::kKLoads + L::kVLoads>();
        else if (!last) wait_vm<L::kKLoads + L::kVLoads>();
        else wait_vm<0>();
      } else {
        if (more) wait_vm<L::kKLoads>();
        else wait_vm<0>();
      }
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      sums(slot);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);
      __builtin_amdgcn_sched_barrier(0);
      if (more) issue_values(after, slot);
      now = next;
      next = L::kSlots == 2 ? after : unit_of(s + 2 * kStride);
      if (L::kSlots == 2) slot ^= 1;
    }

    // ---- results: o - corr, joined over columns and wavefronts, then out or the workspace
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] = sum_over_quads(l[n]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float own = PK == 1 ? corr[n][g][0] : __shfl(corr[n][g][0], r + 16 * (4 / PK) * bank, kWave);
        const float grown = 1.0f / static_cast<float>(shrink[n][g][0]);
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][g][y][i] = (o[n][g][y][i] - own) * grown;
      }
    }
    // channel of row 4 kb + i of tile y of group g
    auto channel = [&](int g, int y, int i) {
      const int q = 4 * kb + i;
      if constexpr (GROUP == 128) return g * 128 + 8 * q + (y < 4 ? 2 * y : 2 * y - 7);
      else if constexpr (GROUP == 64) return g * 64 + 8 * (q & 7) + 2 * y + (q >> 3);
      else return g * 32 + 8 * (q & 3) + 4 * ((q >> 2) & 1) + 2 * y + (q >> 3);
    };
    constexpr int kPad = L::kPad;
    {
      // 16 columns at a time: maxima and sums of every wavefront, then their scaled sums
      float* all = reinterpret_cast<float*>(lds);
      float* stat = all + kWaves * 16 * kPad;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        __syncthreads();
        if (kb == 0) {
          stat[wave * 32 + r] = base[n];
          stat[wave * 32 + 16 + r] = l[n];
        }
        __syncthreads();
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWaves * PK; ++w)
          mm = fmaxf(mm, stat[(w / PK) * 32 + (w % PK) * L::kCols + r % L::kCols]);
        const float f = base[n] == -INFINITY ? 0.0f : exp2_fast(base[n] - mm);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) all[(wave * 16 + r) * kPad + channel(g, y, i)] = o[n][g][y][i] * f;
        __syncthreads();
        // 4 channels of a row at a time
        for (int at = threadIdx.x; at < L::kCols * (D / 4); at += 256) {
          const int rr = at / (D / 4), c0 = at % (D / 4) * 4;
          const int row = row_lo + 16 * n + rr;
          if (row >= rows) continue;
          float M = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves * PK; ++w) M = fmaxf(M, stat[(w / PK) * 32 + (w % PK) * L::kCols + rr]);
          f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < kWaves * PK; ++w) {
            const int col = (w % PK) * L::kCols + rr;
            const float m = stat[(w / PK) * 32 + col];
            sum += sum_at(stat[(w / PK) * 32 + 16 + col], m, M);
            v += *reinterpret_cast<const f32x4*>(all + ((w / PK) * 16 + col) * kPad + c0);
          }
          const int tok = row / a.ratio;
          const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + kvh * a.ratio + row - tok * a.ratio;
          if (chunks > 1 || item.shared) {
            const int64_t at = slot_of<PART>(a, rh, split);
            *reinterpret_cast<f32x4*>(a.part_o + at * D + c0) = v;
            if (c0 == 0) a.part_ml[at] = make_float2(M, sum);
          } else {
            v *= inverse_of(sum);
            *reinterpret_cast<u32x2*>(a.out + rh * D + c0) = u32x2{pack_pair<DT>(v.x, v.y), pack_pair<DT>(v.z, v.w)};
            if (a.lse && c0 == 0) a.lse[rh] = lse_of(M, sum);
          }
        }
      }
    }
    __syncthreads();   // LDS is free for the next rows
  }
}

// Two blocks a compute unit or more, in ordinary registers alone (in the
// accumulator form every round copied the sums out and back for the test of
// the maximum: 35 instead of 25 us for 7 sequences of 32 heads in groups of
// 32), where the sums (NT D / 16) and a group's products and scales fit 256.
constexpr int attention_occupancy(int D, int group, int pk, int nt) { return nt * D + 16 * (D / group) * pk * nt <= 320 ? 2 : 1; }
template <int DT, int D, int GROUP, int PK, int NT>
__global__ __launch_bounds__(256, attention_occupancy(D, GROUP, PK, NT)) void attention_kernel(AttnArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * Shape<D, GROUP, PK, NT>::kWaveBytes];
  attention_block<DT, D, GROUP, PK, NT, kWhole>(a, blockIdx.x, lds);
}

// Joins the chunks of rows whose keys were split: a block a row and head,
// D / 4 threads of four channels for each of 1024 / D chunks at a time.
template <int DT, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int rows_per_tile) {
  constexpr int kWide = D / 4, kGroups = 256 / kWide;
  __shared__ f32x4 sums[256];
  const int lane = threadIdx.x & (kWave - 1);
  const int part = threadIdx.x / kWide, c4 = threadIdx.x % kWide;
  const int h = blockIdx.y, b = blockIdx.z;
  const Sequence sq = sequence_of(a, b);
  for (int i = blockIdx.x; i < sq.n; i += gridDim.x) {
    const int tile = (i * a.ratio + h % a.ratio) / rows_per_tile;
    const int lo = sq.first + tile * rows_per_tile / a.ratio;
    const int hi = sq.first + (min((tile + 1) * rows_per_tile, sq.n * a.ratio) - 1) / a.ratio;
    const int chunks = (steps_of(a, lo, hi).count + a.chunk - 1) / a.chunk;
    if (chunks <= 1) continue;
    const int64_t rh = static_cast<int64_t>(sq.row0 + i) * a.q_heads + h;
    const float2* ml = a.part_ml + rh * a.splits;
    float m = -INFINITY, l = 0.0f;
    for (int c = lane; c < chunks; c += kWave) m = fmaxf(m, ml[c].x);
    m = wave_max(m);
    for (int c = lane; c < chunks; c += kWave) l += sum_at(ml[c].y, ml[c].x, m);
    l = wave_sum(l);
    f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = part; c < chunks; c += kGroups) {
      const float mc = ml[c].x;
      const float f = mc == -INFINITY ? 0.0f : exp2_fast(mc - m);
      o += *reinterpret_cast<const f32x4*>(a.part_o + (rh * a.splits + c) * D + 4 * c4) * f;
    }
    __syncthreads();
    sums[threadIdx.x] = o;
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) o += sums[g * kWide + c4];
      o *= inverse_of(l);
      *reinterpret_cast<u32x2*>(a.out + rh * D + 4 * c4) = u32x2{pack_pair<DT>(o.x, o.y), pack_pair<DT>(o.z, o.w)};
      if (a.lse && c4 == 0) a.lse[rh] = lse_of(m, l);
    }
  }
}

// The same for a batch with shared prefixes: the chunks of the prefix, then the
// sequence's own (rows of one chunk and no prefix have their results).
template <int DT, int D>
__global__ __launch_bounds__(256) void attention_join_parts_kernel(SharedArgs a) {
  constexpr int kWide = D / 4, kGroups = 256 / kWide;
  __shared__ f32x4 sums[256];
  const int lane = threadIdx.x & (kWave - 1);
  const int part = threadIdx.x / kWide, c4 = threadIdx.x % kWide;
  const int h = blockIdx.y, b = blockIdx.z;
  const Item item = own_item(a, b);
  const int own = part_chunks<kOwn>(a, item).chunks;
  const int before = item.shared ? chunks_of(steps_in(item.lo), a.p_splits, a.p_least, a.p_round).chunks : 0;
  const int chunks = before + own;
  if (!item.shared && own <= 1) return;
  for (int i = blockIdx.x; i < item.sq.n; i += gridDim.x) {
    const int64_t rh = static_cast<int64_t>(item.sq.row0 + i) * a.q_heads + h;
    const int64_t first = rh * (a.p_splits + a.splits);
    auto slot = [&](int c) { return first + (c < before ? c : a.p_splits + c - before); };
    float m = -INFINITY, l = 0.0f;
    for (int c = lane; c < chunks; c += kWave) m = fmaxf(m, a.part_ml[slot(c)].x);
    m = wave_max(m);
    for (int c = lane; c < chunks; c += kWave) {
      const float2 ml = a.part_ml[slot(c)];
      l += sum_at(ml.y, ml.x, m);
    }
    l = wave_sum(l);
    f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = part; c < chunks; c += kGroups) {
      const int64_t at = slot(c);
      const float mc = a.part_ml[at].x;
      const float f = mc == -INFINITY ? 0.0f : exp2_fast(mc - m);
      o += *reinterpret_cast<const f32x4*>(a.part_o + at * D + 4 * c4) * f;
    }
    __syncthreads();
    sums[threadIdx.x] = o;
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) o += sums[g * kWide + c4];
      o *= inverse_of(l);
      *reinterpret_cast<u32x2*>(a.out + rh * D + 4 * c4) = u32x2{pack_pair<DT>(o.x, o.y), pack_pair<DT>(o.z, o.w)};
      if (a.lse && c4 == 0) a.lse[rh] = lse_of(m, l);
    }
  }
}

// And for many rows: a wavefront to a row, whose lanes hold the chunks' statistics,
// so that nothing waits for a block and all rows are there at once.  324 x 16 rows
// of 64 channels 10.2 -> 7 us; but few rows of many chunks need the block: 30000
// tokens of 4 beams 32 us whole, 40 with this.
template <int DT, int D>
__global__ __launch_bounds__(256) void attention_join_rows_kernel(SharedArgs a) {
  constexpr int kWide = D / 4, kParts = kWave / kWide;         // lanes to a chunk, chunks at once
  const int lane = threadIdx.x & (kWave - 1);
  const int part = lane / kWide, c4 = lane % kWide;
  const int h = static_cast<int>(blockIdx.y) * kWaves + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const Item item = own_item(a, blockIdx.z);
  const int own = part_chunks<kOwn>(a, item).chunks;
  const int before = item.shared ? chunks_of(steps_in(item.lo), a.p_splits, a.p_least, a.p_round).chunks : 0;
  const int chunks = before + own;
  if (h >= a.q_heads || (!item.shared && own <= 1)) return;
  for (int i = blockIdx.x; i < item.sq.n; i += gridDim.x) {
    const int64_t rh = static_cast<int64_t>(item.sq.row0 + i) * a.q_heads + h;
    const int64_t first = rh * (a.p_splits + a.splits);
    auto slot = [&](int c) { return first + (c < before ? c : a.p_splits + c - before); };
    float m = -INFINITY, l = 0.0f;
    for (int c = lane; c < chunks; c += kWave) m = fmaxf(m, a.part_ml[slot(c)].x);
    m = wave_max(m);
    f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c0 = 0; c0 < chunks; c0 += kWave) {
      const float2 ml = c0 + lane < chunks ? a.part_ml[slot(c0 + lane)] : make_float2(-INFINITY, 0.0f);
      const float weight = ml.x == -INFINITY ? 0.0f : exp2_fast(ml.x - m);
      l += sum_at(ml.y, ml.x, m);
      const int n = min(chunks - c0, kWave);
      for (int c = 0; c < n; c += kParts) {        // (eight loads at once gained nothing)
        const float f = __shfl(weight, min(c + part, kWave - 1), kWave);
        if (c + part < n) o += *reinterpret_cast<const f32x4*>(a.part_o + slot(c0 + c + part) * D + 4 * c4) * f;
      }
    }
    l = wave_sum(l);
#pragma unroll
    for (int lanes = kWide; lanes < kWave; lanes *= 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], lanes, kWave);
    if (part == 0) {
      o *= inverse_of(l);
      *reinterpret_cast<u32x2*>(a.out + rh * D + 4 * c4) = u32x2{pack_pair<DT>(o.x, o.y), pack_pair<DT>(o.z, o.w)};
      if (a.lse && c4 == 0) a.lse[rh] = lse_of(m, l);
    }
  }
}

}  // namespace
}  // namespace qmm
