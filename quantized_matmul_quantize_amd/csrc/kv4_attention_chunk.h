// kv4_attention_chunk.h -- the attention kernel for chunks of queries (see
// kv4_attention.h for the products and their operand layouts).
//
// With many rows the operations that make operands of codes would outweigh the
// products, so the wavefronts of a block, each with rows of its own, share
// them: per round of keys two wavefronts expand keys, two values, subtract the
// zero-points (c - z is exact in binary16) and leave whole matrix-core operands
// in LDS for the next round, while all compute on those of the round before:
// one barrier a round.  What is left per score is one multiplication by the
// key's scale (with the running base in the same operation where a head is one
// group), the exponential, a conversion and half a packed product with the
// value's scale, and the sum of the probabilities (on the matrix cores it would
// be the sum of their roundings, 10^-4 off where a row sees few keys).
// (The power of two of bf16 queries is the block's.)  Three chunks of 2048
// queries on 8192 keys, 32 and 8 heads of 128 in one group: 605 GFLOP in 855
// us, 708 TFLOP/s, 60% of what a large bf16 product of the library reaches (with
// powers of two shared by the rows of a tile 834 us, but a hidden token's scale
// then cost other rows their bits); in groups of 64 each operand is read for one
// tile of rows only, 2 x 1024 queries on 6000 keys 216 us, 403 TFLOP/s; two
// wavefronts a SIMD (the sums hold the registers) leave part of the LDS latency
// and of the exponentials uncovered.
#pragma once

#include "kv4_attention.h"

namespace qmm {
namespace {

template <int D, int GROUP, int NT>
struct Chunk {
  static constexpr int kG = D / GROUP;
  static constexpr int kRows = 16 * NT * kWaves;
  static constexpr int kKeys = D == 256 ? 32 : 64;          // of a round
  static constexpr int kSteps = D / 32;
  // operands of 1 KiB: [16-key tile][k-extent] of keys, [step][16 channels] of values; two buffers of each
  static constexpr int kKOps = kKeys / 16 * kSteps, kVOps = kKeys / kStep * (D / 16);
  static constexpr int kVStride = 1024 + 80;                // a value's eight channels go to 16 operand rows: no bank twice
  static constexpr int kKScales = kKOps * 1024;             // fp32 [group][key]
  static constexpr int kKBuffer = kKScales + kG * kKeys * 4;
  static constexpr int kVScales = kVOps * kVStride;         // binary16 [group][key]
  static constexpr int kVBuffer = kVScales + kG * kKeys * 2;
  static_assert(kKBuffer % 16 == 0 && kVBuffer % 16 == 0, "alignment");
  // what a lane expands of a round: kWords words of a key's codes; of a word of two quads of values kNibbles
  // nibbles of either its low or its high half (kShare lanes a word)
  static constexpr int kWords = kKeys * D / (512 * kWaves), kKeyWaves = D / (32 * kWords);
  static constexpr int kShare = 64 * kWaves / (kKeys * D / 64), kNibbles = 8 / kShare;
};

// Lane (r, kb) finds its 16 bytes of an operand in lane order, and producers
// are mapped so that any 16 lanes write 16 different rows: no bank conflicts.
__device__ __forceinline__ int op_at(int r, int kb) { return 16 * (16 * kb + r); }

template <int DT, int D, int GROUP, int NT>
__device__ __forceinline__ void attention_chunk_block(const AttnArgs& a) {
  using L = Chunk<D, GROUP, NT>;
  constexpr int G = L::kG, MT = GROUP / 16, KEYS = L::kKeys, kSteps = L::kSteps;
  constexpr int U = KEYS / kStep;                  // steps of a round
  constexpr int kTiles = KEYS / 16;                // 16-key tiles of a round
  constexpr int kWords = L::kWords;
  constexpr int kAhead = 2;                        // operands read before they are used
  constexpr int kAluMayCross = 0x6;                // sched_barrier: scalar and vector arithmetic
  __shared__ __attribute__((aligned(16))) uint8_t k_lds[2][L::kKBuffer];
  __shared__ __attribute__((aligned(16))) uint8_t v_lds[2][L::kVBuffer];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r = lane & 15, kb = lane >> 4;
  uint32_t id = blockIdx.x;
  const int kvh = static_cast<int>(id % a.sh.heads);
  id /= a.sh.heads;
  const int split = static_cast<int>(id % a.splits);
  id /= a.splits;
  const int b = static_cast<int>(id % a.seqs);
  const int order = static_cast<int>(id / a.seqs);
  const Sequence sq = sequence_of(a, b);
  const int rows = sq.n * a.ratio;
  const int tiles = (rows + L::kRows - 1) / L::kRows;
  const int record = static_cast<int>(a.sh.record_bytes());
  const uint32_t page_bytes = static_cast<uint32_t>(a.sh.heads) * static_cast<uint32_t>(record);
  const uint32_t pages = static_cast<uint32_t>(a.sh.pages);
  const uint8_t* head = a.cache + static_cast<int64_t>(kvh) * record;
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const table_t table = (table_t)(a.table + b * a.table_stride);

  // What a lane expands of a round.  Keys: kWords words of key r of a 16-key
  // tile (kKeyWaves wavefronts a tile).  Values: of one word of both quads
  // `v_quad` of a step half the channels (`part`: even or odd ones) or a
  // quarter.
  const int k_tile = wave / L::kKeyWaves;
  const int k_piece = 4 * (wave % L::kKeyWaves) + kb;               // of 4 kWords bytes
  const int v_unit = 64 * (wave / L::kShare) + lane;
  const int v_word = v_unit % (D / 8), v_quad = v_unit / (D / 8) % 4;
  const int v_step = D == 64 ? v_unit >> 5 : U == 2 ? wave / L::kShare : 0;
  const int part = wave % L::kShare & 1, v_first = L::kNibbles * (wave % L::kShare >> 1);   // first of its nibbles
  const int v_group = v_word / (GROUP / 8);
  const int k_at = r * (D / 2) + 4 * kWords * k_piece, kp_at = a.sh.page * D + 4 * r;
  const int v_at = a.sh.page * (D / 2) + 16 * v_word + v_quad * (2 * D);
  const int vp_at = a.sh.page * (D + 4 * G) + v_group * a.sh.page * 4 + 16 * v_quad;

  // the last tiles see the most keys and go first
  for (int tile = tiles - 1 - order; tile >= 0; tile -= a.row_tiles) {
    const int blk_last = min((tile + 1) * L::kRows, rows) - 1;
    const int blk_lo = sq.first + tile * L::kRows / a.ratio, blk_hi = sq.first + blk_last / a.ratio;
    const Steps st = steps_of(a, blk_lo, blk_hi);
    const int chunks = max(1, (st.count + a.chunk - 1) / a.chunk);
    if (split >= chunks) continue;
    const int s_lo = split * a.chunk, s_hi = min(s_lo + a.chunk, st.count);
    const int rounds = (s_hi - s_lo + U - 1) / U;
    // Keys that no row of the block sees: past blk_hi, in the last round, or up to
    // `hide` and no sinks, in the step where the window begins and the one before
    // (rounds that hold them are cleaned, and the sinks' with them).
    const int hide = a.window > 0 ? blk_lo - a.window : -1;
    const int row_lo = tile * L::kRows + wave * 16 * NT;
    const int row_hi = min(row_lo + 16 * NT, rows) - 1;
    const int pos_lo = sq.first + row_lo / a.ratio;
    const int pos_hi = row_hi < row_lo ? -1 : sq.first + row_hi / a.ratio;

    // ---- queries: second operands, the block's power of two, positions
    u32x4 qv[NT][kSteps];
    int pos[NT];
    float most = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row_lo + 16 * n + r;
      const bool live = row < rows;
      const int tok = live ? row / a.ratio : 0, qh = live ? kvh * a.ratio + row - tok * a.ratio : 0;
      pos[n] = live ? sq.first + tok : -1;
      const uint16_t* qp = a.q + (sq.row0 + tok) * a.q_ts + qh * a.q_hs + 8 * kb;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) qv[n][j] = live ? ld16(qp + 32 * j) : u32x4{0u, 0u, 0u, 0u};
      if constexpr (DT == QMM_BF16) most = largest_bf16(qv[n], most);
    }
    float unscale = 1.0f;
    __syncthreads();                               // LDS is free: the rows before are done
    if constexpr (DT == QMM_BF16) {
      float* stat = reinterpret_cast<float*>(&k_lds[0][0]);
      most = wave_max(most);
      if (lane == 0) stat[wave] = most;
      __syncthreads();
      most = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) most = fmaxf(most, stat[w]);
      const QueryScale qs = query_scale(most);
      __syncthreads();
      unscale = qs.up;
#pragma unroll
      for (int n = 0; n < NT; ++n) to_f16(qv[n], qs.down);
    }
    const float key_scale = a.scale_log2 * unscale;

    // ---- rounds: first keys of their steps, pages of their tiles
    struct Round {
      int key[U], page[kTiles];
    };
    auto round_of = [&](int round) {
      Round x;
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const int at = s_lo + round * U + c;
        x.key[c] = at < s_hi ? st.key(at) : kBeyond;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = x.key[c] + 16 * u;
          const int page = table[max(min(t, sq.ctx - 1), 0) >> a.sh.shift];
          x.page[2 * c + u] = t < sq.ctx ? page : -1;
        }
      }
      return x;
    };
    auto holes_of = [&](const Round& x) {
      int h = 0;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) h |= static_cast<uint32_t>(x.page[t]) < pages ? 0 : 1 << t;
      return h;
    };
    // A 16-key tile past the context, or whose page is not of this cache, is
    // read through an empty resource: zeros, so scales of 0.
    auto tile_of = [&](int page) {
      const bool here = static_cast<uint32_t>(page) < pages;
      return __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(head + static_cast<uint64_t>(static_cast<uint32_t>(here ? page : 0)) * page_bytes), 0,
          here ? record : 0, kBufferWord3);
    };
    // ---- producers
    uint32_t k_raw[kWords], k_par[G];
    u32x4 v_raw[2], v_par[2];
    // first key of the wavefront's tile of keys, and its page
    struct Mine {
      int key, page;
    };
    auto mine_of = [&](int round) {
      const int at = s_lo + round * U + (U == 1 ? 0 : k_tile >> 1);
      Mine x;
      x.key = (at < s_hi ? st.key(at) : kBeyond) + 16 * (k_tile & 1);
      const int page = table[max(min(x.key, sq.ctx - 1), 0) >> a.sh.shift];
      x.page = x.key < sq.ctx ? page : -1;
      return x;
    };
    auto fetch_keys = [&](Mine x) {
      const int t0 = x.key;
      const __amdgpu_buffer_rsrc_t rs = tile_of(x.page);
      const int place = t0 & (a.sh.page - 1);
      if constexpr (kWords == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, k_at, place * (D / 2), 0));
        k_raw[0] = v.x;
        k_raw[1] = v.y;
      } else {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, k_at, place * (D / 2), 0));
#pragma unroll
        for (int w = 0; w < 4; ++w) k_raw[w] = v[w];
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
        k_par[g] = __builtin_amdgcn_raw_buffer_load_b32(rs, kp_at + g * a.sh.page * 4, place * 4, 0);
    };
    // The memory of hidden keys may hold anything.  Scores are replaced whatever
    // they are (past the context, where rows that are none may not be masked,
    // the keys' scales are taken as 0); but 0 times a scale that is a NaN would
    // be one, so of a key that no row of the block sees the values' scale is
    // taken as 0.
    auto clean_keys = [&](Mine x) {
#pragma unroll
      for (int g = 0; g < G; ++g) k_par[g] = x.key + r < sq.ctx ? k_par[g] : 0u;
    };
    auto fetch_values = [&](const Round& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < U; ++c) {
          // D 128: the wavefront's step; D 64: the steps of its halves
          if (D == 64 ? v_step == c : U == 1 || v_step == c) {
            const __amdgpu_buffer_rsrc_t rs = tile_of(x.page[2 * c + i]);
            const int place = (x.key[c] + 16 * i) & (a.sh.page - 1);
            v_raw[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, v_at, place * (D / 2), 0));
            v_par[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, vp_at, place * 4, 0));
          }
        }
    };
    auto clean_values = [&](const Round& x) {
      int t0 = x.key[0];
#pragma unroll
      for (int c = 1; c < U; ++c) t0 = v_step == c ? x.key[c] : t0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + 16 * i + 4 * v_quad + e;
          v_par[i][e] = t <= blk_hi && (t > hide || t < a.sinks) ? v_par[i][e] : 0u;
        }
    };
    const uint32_t magic = vgpr_const(Codes64::magic);
    auto less = [](uint32_t p, uint32_t z) {       // pairs: (64 + c) + -(64 + z)
      return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, p) + __builtin_bit_cast(f16x2_t, z));
    };
    auto expand_keys = [&](uint8_t* buf) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const int word = kWords * k_piece + w;     // k-extent j of lane quarter kb is word kSteps kb + j
        const int j = kWords == kSteps ? w : word % kSteps;
        uint32_t par = k_par[0];
#pragma unroll
        for (int g = 1; g < G; ++g) par = j * 32 / GROUP == g ? k_par[g] : par;
        const uint32_t z = 0xD400D400u + ((par >> 16) & 0xFu) * 0x00100010u;
        uint32_t p[4];
        Codes64::unpack(k_raw[w], magic, p);
        *reinterpret_cast<u32x4*>(buf + (k_tile * kSteps + j) * 1024 + op_at(r, word / kSteps)) =
            u32x4{less(p[0], z), less(p[1], z), less(p[2], z), less(p[3], z)};
      }
      if (k_piece == 0) {
#pragma unroll
        for (int g = 0; g < G; ++g)
          *reinterpret_cast<float*>(buf + L::kKScales + (g * KEYS + 16 * k_tile + r) * 4) =
              kv4_scale(k_par[g]) * key_scale;
      }
    };
    auto expand_values = [&](uint8_t* buf) {
      uint32_t z[4], w[4];
      const uint32_t sel = part ? 0x07060302u : 0x05040100u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[e] = (__builtin_amdgcn_perm(v_par[e >> 1][2 * (e & 1) + 1], v_par[e >> 1][2 * (e & 1)], 0x0c060c02u) << 4 &
                0x00F000F0u) | 0xD400D400u;
        w[e] = __builtin_amdgcn_perm(v_raw[e >> 1][2 * (e & 1) + 1], v_raw[e >> 1][2 * (e & 1)], sel) >> (4 * v_first);
      }
#pragma unroll
      for (int y = 0; y < L::kNibbles; ++y) {
        u32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = less(((y == 0 ? w[e] << 4 : w[e] >> (4 * y - 4)) & Codes64::mask) | magic, z[e]);
        const int row = 8 * (v_word & 1) + 2 * (v_first + y) + part;
        *reinterpret_cast<u32x4*>(buf + (v_step * (D / 16) + v_word / 2) * L::kVStride + op_at(row, v_quad)) = v;
      }
      if (part == 0 && v_first == 0 && v_word % (GROUP / 8) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<u32x2*>(buf + L::kVScales + (v_group * KEYS + v_step * kStep + 16 * i + 4 * v_quad) * 2) =
              u32x2{__builtin_amdgcn_perm(v_par[i][1], v_par[i][0], 0x05040100u),
                    __builtin_amdgcn_perm(v_par[i][3], v_par[i][2], 0x05040100u)};
      }
    };

    f32x4 o[NT][G][MT];
    float l[NT];           // of this lane's keys
    float base[NT];
    f16x2_t shrink[NT][G]; // the column's, twice
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      base[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        shrink[n][g] = pair16(32768.0f);
#pragma unroll
        for (int y = 0; y < MT; ++y) o[n][g][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }

    // Scores of a round, less the base they were taken at (0 before the first
    // key): products of c - z, then the keys' scales, the base in the same
    // operation.
    f32x4 x[NT][2 * U];
    float from[NT], limit[NT];                     // the base or 0; where the maximum has to move
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      from[n] = 0.0f;
      limit[n] = -INFINITY;
    }
    auto scores = [&](const uint8_t* buf, f32x4 (&to)[NT][2 * U]) {
      constexpr int kOps = 2 * U * kSteps;
      u32x4 k[kAhead];
      auto read = [&](int i) { return *reinterpret_cast<const u32x4*>(buf + i * 1024 + op_at(r, kb)); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) k[i] = read(i);
      __builtin_amdgcn_sched_barrier(kAluMayCross);
      f32x4 acc[NT];
#pragma unroll
      for (int i = 0; i < kOps; ++i) {
        const int u = i / kSteps, j = i % kSteps, g = j * 32 / GROUP;
        if (j * 32 % GROUP == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n] = mfma(k[i % kAhead], qv[n][j], acc[n]);
        if (i + kAhead < kOps) k[i % kAhead] = read(i + kAhead);
        __builtin_amdgcn_sched_barrier(kAluMayCross);
        if ((j + 1) * 32 % GROUP == 0) {
          const f32x4 sc = *reinterpret_cast<const f32x4*>(buf + L::kKScales + (g * KEYS + 16 * u + 4 * kb) * 4);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) to[n][u][e] = fmaf(acc[n][e], sc[e], g == 0 ? -from[n] : to[n][u][e]);
        }
      }
    };
    float top[NT];
    bool hides;            // some key from some row
    // masks of a round's scores, their maxima
    auto mask = [&](const Round& now) {
      const int first = now.key[0], end = now.key[U - 1] + kStep, holes = holes_of(now);
      const bool whole = holes == 0 && end - first == U * kStep && end - 1 <= pos_lo &&
                         (a.window == 0 || first > pos_hi - a.window || end <= a.sinks);
      hides = !whole;
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
          const bool here = !((holes >> u) & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = now.key[u / 2] + 16 * (u % 2) + 4 * kb + i;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const bool seen = here && t <= pos[n] && (a.window == 0 || t > pos[n] - a.window || t < a.sinks);
              x[n][u][i] = seen ? x[n][u][i] : -INFINITY;
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float t = max3(x[n][0][0], x[n][0][1], x[n][0][2]);
        t = max3(t, x[n][0][3], x[n][1][0]);
        t = max3(t, x[n][1][1], x[n][1][2]);
        if constexpr (U == 1) {
          t = max3(t, x[n][1][3], x[n][1][3]);
        } else {
          t = max3(t, x[n][1][3], x[n][2][0]);
          t = max3(t, x[n][2][1], x[n][2][2]);
          t = max3(t, x[n][2][3], x[n][3][0]);
          t = max3(t, x[n][3][1], x[n][3][2]);
          t = max3(t, x[n][3][3], x[n][3][3]);
        }
        top[n] = t;
      }
    };

    // ---- rounds.  Of round n its scores are taken (and its keys' operands
    // replaced) in round n - 1, its sums in round n: while the scores of the
    // next round are in the matrix cores the vector unit takes this one's
    // exponentials, and under the sums it expands the keys of the round after
    // next and the values of the next.  One barrier a round.
    Round next = round_of(1), third = round_of(2);
    Mine k_now = mine_of(2), k_next = mine_of(3);   // of the keys that are on their way, and of the ones after
    if (rounds > 0) {
      const Round first = round_of(0);
      const Mine k0 = mine_of(0), k1 = mine_of(1);
      fetch_keys(k0);
      fetch_values(first);
      clean_keys(k0);
      clean_values(first);
      expand_keys(&k_lds[0][0]);
      expand_values(&v_lds[0][0]);
      fetch_keys(k1);
      fetch_values(next);
      clean_keys(k1);
      expand_keys(&k_lds[1][0]);
      fetch_keys(k_now);
      __syncthreads();
      scores(&k_lds[0][0], x);
      mask(first);
      __syncthreads();                             // the keys of round 0 may be replaced
    }
    for (int round = 0; round < rounds; ++round) {
      const uint8_t* vb = &v_lds[round & 1][0];
      const Round fourth = round_of(round + 3);
      const Mine k_fifth = mine_of(round + 4);
      // ---- the largest scale of the values, of every second key; the scales
      // themselves are read again where they are used
      auto pairs_of = [&](int g, int u) {          // two pairs of keys
        return *reinterpret_cast<const u32x2*>(vb + L::kVScales + (g * KEYS + 16 * u + 4 * kb) * 2);
      };
      f16x2_t most_s[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        most_s[g] = f16x2_t{0, 0};
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
          const u32x2 v = pairs_of(g, u);
          const uint32_t v0 = v.x, v1 = v.y;
          most_s[g] = pk_max(most_s[g], pk_max(__builtin_bit_cast(f16x2_t, v0), __builtin_bit_cast(f16x2_t, v1)));
        }
      }
      // ---- running maximum and powers of two: one test for both.  What is hidden
      // from a row, such as a later token, must not cost it bits.
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        grow |= top[n] > limit[n];
#pragma unroll
        for (int g = 0; g < G; ++g) grow |= past_one(most_s[g] * shrink[n][g]);
      }
      if (__any(grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float to = fmaxf(base[n], max_over_quads(top[n]) + from[n] - 7.0f);
          const float fade = to == -INFINITY ? 1.0f : exp2_fast(base[n] - to);
          const float now_from = to == -INFINITY ? 0.0f : to;
          f16x2_t own[G];
#pragma unroll
          for (int g = 0; g < G; ++g) own[g] = most_s[g];
          if (hides) {
#pragma unroll
            for (int g = 0; g < G; ++g) own[g] = f16x2_t{0, 0};
#pragma unroll
            for (int u = 0; u < 2 * U; ++u) {
              uint32_t keep[2];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                keep[i] = (x[n][u][2 * i] == -INFINITY ? 0u : 0xFFFFu) |
                          (x[n][u][2 * i + 1] == -INFINITY ? 0u : 0xFFFF0000u);
#pragma unroll
              for (int g = 0; g < G; ++g) {
                const u32x2 v = pairs_of(g, u);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t seen = v[i] & keep[i];
                  own[g] = pk_max(own[g], __builtin_bit_cast(f16x2_t, seen));
                }
              }
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float now_shrink = static_cast<float>(shrink[n][g][0]);
            const float next_shrink = fminf(fminf(now_shrink, shrink_for(max_over_quads(larger(own[g])))),
                                            shrink_for_hidden(max_over_quads(larger(most_s[g]))));
            const float f = fade * (next_shrink / now_shrink);
            shrink[n][g] = pair16(next_shrink);
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= f;
          }
#pragma unroll
          for (int u = 0; u < 2 * U; ++u) x[n][u] += from[n] - now_from;
          from[n] = now_from;
          limit[n] = to == -INFINITY ? -INFINITY : 15.0f;
          base[n] = to;
          l[n] *= fade;
        }
      }
      // ---- the next round's scores, this one's probabilities.  Where the output
      // is bf16 (2^-8 of it) they are rounded to binary16 here and once more with
      // the values' scale, 2^-10 of a row's mass: held in fp32 until then, three
      // chunks of prompts take 941 instead of 902 us, 2 x 1024 queries on 6000
      // keys in groups of 32 349 instead of 281.  The empty asm keeps a pair's
      // sum and conversion at its exponentials: moved away by the compiler they
      // hold registers, and with the spills a prompt's chunk took 1122 instead of
      // 832 us.
      u32x4 p[NT][U];
      f32x4 ahead[NT][2 * U];
      scores(&k_lds[(round + 1) & 1][0], ahead);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < U; ++c) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f32x4& xs = x[n][2 * c + (e >> 1)];
            xs[2 * (e & 1)] = exp2_fast(xs[2 * (e & 1)]);
            xs[2 * (e & 1) + 1] = exp2_fast(xs[2 * (e & 1) + 1]);
            l[n] += xs[2 * (e & 1)] + xs[2 * (e & 1) + 1];
            if constexpr (DT == QMM_BF16) {
              uint32_t pair = pack_pair<QMM_F16>(xs[2 * (e & 1)], xs[2 * (e & 1) + 1]);
              asm volatile("" : "+v"(l[n]), "+v"(pair));
              p[n][c][e] = pair;
            } else {
              asm volatile("" : "+v"(l[n]));
            }
          }
        }
      }
      if (k_now.key + 16 > sq.ctx) clean_keys(k_now);
      if (s_lo + (round + 1) * U <= st.sink_steps || round + 2 >= rounds) clean_values(next);
      // ---- sums; operands of the next rounds
      {
        constexpr int kOps = U * G * MT;
        u32x4 v[kAhead], pv[NT];
        auto read = [&](int i) { return *reinterpret_cast<const u32x4*>(vb + i * L::kVStride + op_at(r, kb)); };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = read(i);
        __builtin_amdgcn_sched_barrier(kAluMayCross);
#pragma unroll
        for (int i = 0; i < kOps; ++i) {
          const int c = i / (G * MT), g = i / MT % G, y = i % MT;
          if (y == 0) {
            const u32x2 s01 = pairs_of(g, 2 * c), s23 = pairs_of(g, 2 * c + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t se = e < 2 ? s01[e & 1] : s23[e & 1];
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const f16x2_t s2 = __builtin_bit_cast(f16x2_t, se) * shrink[n][g];
                if constexpr (DT == QMM_BF16) {
                  const uint32_t pair = p[n][c][e];
                  pv[n][e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, pair) * s2);
                } else {
                  const f32x4& xs = x[n][2 * c + (e >> 1)];
                  pv[n][e] = weighted(xs[2 * (e & 1)], xs[2 * (e & 1) + 1], s2);
                }
              }
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][g][y] = mfma(v[i % kAhead], pv[n], o[n][g][y]);
          if (i + kAhead < kOps) v[i % kAhead] = read(i + kAhead);
          __builtin_amdgcn_sched_barrier(kAluMayCross);
        }
      }
      expand_keys(&k_lds[round & 1][0]);
      expand_values(&v_lds[(round + 1) & 1][0]);
      fetch_keys(k_next);
      fetch_values(third);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) x[n][u] = ahead[n][u];
      mask(next);
      next = third;
      third = fourth;
      k_now = k_next;
      k_next = k_fifth;
      // only LDS is shared: the codes on their way need not have come
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }

    // ---- results: column r of row 4 kb + i of every tile
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row_lo + 16 * n + r;
      const float sum = sum_over_quads(l[n]);
      if (row >= rows) continue;
      const int tok = row / a.ratio;
      const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + kvh * a.ratio + row - tok * a.ratio;
      const float inv = chunks > 1 ? 1.0f : inverse_of(sum);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float f = inv / static_cast<float>(shrink[n][g][0]);
#pragma unroll
        for (int y = 0; y < MT; ++y) {
          const f32x4 v = o[n][g][y] * f;
          const int c0 = (g * MT + y) * 16 + 4 * kb;
          if (chunks > 1)
            *reinterpret_cast<f32x4*>(a.part_o + (rh * a.splits + split) * D + c0) = v;
          else
            *reinterpret_cast<u32x2*>(a.out + rh * D + c0) = u32x2{pack_pair<DT>(v.x, v.y), pack_pair<DT>(v.z, v.w)};
        }
      }
      if (kb == 0) {
        if (chunks > 1) a.part_ml[rh * a.splits + split] = make_float2(base[n], sum);
        else if (a.lse) a.lse[rh] = lse_of(base[n], sum);
      }
    }
  }
}

// Two blocks a compute unit: one wavefront's products then run under the
// other's exponentials.  (A block of eight wavefronts instead, which expands
// half as much a wavefront: 804 instead of 829 us for three chunks of prompts,
// but half as many blocks.)
template <int DT, int D, int GROUP, int NT>
__global__ __launch_bounds__(256, D / GROUP < 8 ? 2 : 1) void attention_chunk_kernel(AttnArgs a) {
  attention_chunk_block<DT, D, GROUP, NT>(a);
}

}  // namespace
}  // namespace qmm
