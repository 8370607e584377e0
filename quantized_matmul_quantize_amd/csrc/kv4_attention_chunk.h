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
// value's scale; the sums of the probabilities come from the matrix cores too.
// (The power of two of bf16 queries is the block's.)
#pragma once

#include "kv4_attention.h"

namespace qmm {
namespace {

template <int D, int GROUP, int NT>
struct Chunk {
  static constexpr int kG = D / GROUP;
  static constexpr int kRows = 16 * NT * kWaves;
  static constexpr int kKeys = 8192 / D;                    // of a round: two 16-byte pieces of codes a producing lane
  static constexpr int kSteps = D / 32;
  // operands of 1 KiB: [16-key tile][k-extent] of keys, [step][16 channels] of values
  static constexpr int kKOps = kKeys / 16 * kSteps, kVOps = kKeys / kStep * (D / 16);
  static constexpr int kVStride = 1024 + 80;                // a value's eight channels go to 16 operand rows: no bank twice
  static constexpr int kVAt = kKOps * 1024;
  static constexpr int kKScales = kVAt + kVOps * kVStride;  // fp32 [group][key]
  static constexpr int kVScales = kKScales + kG * kKeys * 4;  // binary16 [group][key]
  static constexpr int kBuffer = kVScales + kG * kKeys * 2;
  static_assert(kBuffer % 16 == 0, "alignment");
};

// Lane (r, kb) finds its 16 bytes of an operand in lane order, and producers
// are mapped so that any 16 lanes write 16 different rows: no bank conflicts.
__device__ __forceinline__ int op_at(int r, int kb) { return 16 * (16 * kb + r); }

template <int DT, int D, int GROUP, int NT>
__device__ __forceinline__ void attention_chunk_block(const AttnArgs& a) {
  using L = Chunk<D, GROUP, NT>;
  constexpr int G = L::kG, MT = GROUP / 16, KEYS = L::kKeys, kSteps = L::kSteps;
  constexpr int kPer = KEYS / kStep;               // steps of a round
  constexpr int kPieces = D / 32;                  // 16-byte pieces of a key
  constexpr int kTiles = KEYS / 16;                // 16-key tiles of a round
  constexpr int U = kPer < 2 ? 1 : 2;              // steps whose scores are taken together
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][L::kBuffer];

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

  // Producers: wavefronts 0 and 1 keys, 2 and 3 values.  Of a round a lane
  // takes two pieces of 16 bytes: of keys the lane's (lane & 15) in one or two
  // 16-key tiles, or of both tiles of a step the same word of the same quad of
  // keys.
  const bool values = wave >= 2;
  const int half = wave & 1;
  const int unit = 64 * half + lane;
  const int v_word = unit % (D / 8), v_quad = unit / (D / 8) % 4, v_step = unit / (D / 2);
  const int v_group = v_word / (GROUP / 8);
  int k_piece[2], my_tile[2];                      // my_tile: the 16-key tile of a piece
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int m = 4 * (2 * i + half) + (lane >> 4);
    k_piece[i] = m % kPieces;
    my_tile[i] = values ? 2 * v_step + i : m / kPieces;
  }
  const int first_key = values ? 4 * v_quad : r;   // of the lane's in a tile
  // byte offsets in a record: at + place * per (codes), params likewise
  const int raw_at = values ? a.sh.page * (D / 2) + 16 * v_word + v_quad * (2 * D) : r * (D / 2);
  const int par_at = values ? a.sh.page * (D + 4 * G) + v_group * a.sh.page * 4 + 16 * v_quad : a.sh.page * D + 4 * r;

  // the last tiles see the most keys and go first
  for (int tile = tiles - 1 - order; tile >= 0; tile -= a.row_tiles) {
    const int blk_last = min((tile + 1) * L::kRows, rows) - 1;
    const Steps st = steps_of(a, sq.first + tile * L::kRows / a.ratio, sq.first + blk_last / a.ratio);
    const int chunks = max(1, (st.count + a.chunk - 1) / a.chunk);
    if (split >= chunks) continue;
    const int s_lo = split * a.chunk, s_hi = min(s_lo + a.chunk, st.count);
    const int rounds = (s_hi - s_lo + kPer - 1) / kPer;
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
      float* stat = reinterpret_cast<float*>(&lds[0][0]);
      most = wave_max(most);
      if (lane == 0) stat[wave] = most;
      __syncthreads();
      const QueryScale qs = query_scale(fmaxf(fmaxf(stat[0], stat[1]), fmaxf(stat[2], stat[3])));
      __syncthreads();
      unscale = qs.up;
#pragma unroll
      for (int n = 0; n < NT; ++n) to_f16(qv[n], qs.down);
    }
    const float key_scale = a.scale_log2 * unscale;

    // ---- producers
    u32x4 raw[2];
    uint32_t kpar[2][G];                           // keys: params of the two pieces' keys
    u32x4 vpar[2];                                 // values: params of the two quads' keys
    struct Round {                                 // first keys of its steps, pages of its tiles
      int key[kPer], page[kTiles];
    };
    auto round_of = [&](int round) {
      Round x;
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        const int at = s_lo + round * kPer + c;
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
    auto fetch = [&](const Round& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // D 128 and 256: the tile is the wavefront's; D 64: two tiles of 32 lanes each, with a part of the lanes each
        constexpr int kPasses = D == 64 ? 2 : 1;
#pragma unroll
        for (int pass = 0; pass < kPasses; ++pass) {
          const int tile_n = D == 64 ? (values ? 4 * half + 2 * pass + i : 2 * (2 * i + half) + pass)
                             : D == 128 ? (values ? 2 * half + i : 2 * i + half) : i;
          int page = x.page[0], t0 = x.key[0];
#pragma unroll
          for (int t = 1; t < kTiles; ++t) {
            page = tile_n == t ? x.page[t] : page;
            t0 = tile_n == t ? x.key[t / 2] + 16 * (t % 2) : t0;
          }
          if (D != 64 || (lane >> 5) == pass) {
            const bool here = static_cast<uint32_t>(page) < pages;
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint8_t*>(head + static_cast<uint64_t>(static_cast<uint32_t>(here ? page : 0)) * page_bytes),
                0, here ? record : 0, kBufferWord3);
            const int place = t0 & (a.sh.page - 1);
            raw[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   rs, raw_at + (values ? 0 : 16 * k_piece[i]), place * (D / 2), 0));
            if (values) {
              vpar[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, par_at, place * 4, 0));
            } else {
#pragma unroll
              for (int g = 0; g < G; ++g)
                kpar[i][g] = __builtin_amdgcn_raw_buffer_load_b32(rs, par_at + g * a.sh.page * 4, place * 4, 0);
            }
          }
        }
      }
    };
    // Memory past the context may hold anything: its scales and zero-points are taken as 0.
    auto clean = [&](const Round& x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        int t0 = x.key[0];
#pragma unroll
        for (int t = 1; t < kTiles; ++t) t0 = my_tile[i] == t ? x.key[t / 2] + 16 * (t % 2) : t0;
        const int key = t0 + first_key;
#pragma unroll
        for (int e = 0; e < 4; ++e) vpar[i][e] = key + e < sq.ctx ? vpar[i][e] : 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) kpar[i][g] = key < sq.ctx ? kpar[i][g] : 0u;
      }
    };
    const uint32_t magic = vgpr_const(Codes64::magic);
    auto less = [](uint32_t p, uint32_t z) {       // pairs: (64 + c) + -(64 + z)
      return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, p) + __builtin_bit_cast(f16x2_t, z));
    };
    auto expand = [&](uint8_t* buf) {
      if (!values) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int first = 4 * k_piece[i];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = (first + x) % kSteps;    // the word's k-extent and eight channels of it
            uint32_t par = kpar[i][0];
#pragma unroll
            for (int g = 1; g < G; ++g) par = j * 32 / GROUP == g ? kpar[i][g] : par;
            const uint32_t z = 0xD400D400u + ((par >> 16) & 0xFu) * 0x00100010u;
            uint32_t p[4];
            Codes64::unpack(raw[i][x], magic, p);
            *reinterpret_cast<u32x4*>(buf + (my_tile[i] * kSteps + j) * 1024 + op_at(r, (first + x) / kSteps)) =
                u32x4{less(p[0], z), less(p[1], z), less(p[2], z), less(p[3], z)};
          }
          if (k_piece[i] == 0) {
#pragma unroll
            for (int g = 0; g < G; ++g)
              *reinterpret_cast<float*>(buf + L::kKScales + (g * KEYS + 16 * my_tile[i] + r) * 4) =
                  kv4_scale(kpar[i][g]) * key_scale;
          }
        }
      } else {
        uint32_t z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          z[e] = (__builtin_amdgcn_perm(vpar[e >> 1][2 * (e & 1) + 1], vpar[e >> 1][2 * (e & 1)], 0x0c060c02u) << 4 &
                  0x00F000F0u) | 0xD400D400u;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = __builtin_amdgcn_perm(raw[e >> 1][2 * (e & 1) + 1], raw[e >> 1][2 * (e & 1)],
                                         part ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = less(((y == 0 ? w[e] << 4 : w[e] >> (4 * y - 4)) & Codes64::mask) | magic, z[e]);
            const int row = 8 * (v_word & 1) + 2 * y + part;
            *reinterpret_cast<u32x4*>(buf + L::kVAt + (v_step * (D / 16) + v_word / 2) * L::kVStride +
                                      op_at(row, v_quad)) = v;
          }
        }
        if (v_word % (GROUP / 8) == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<u32x2*>(buf + L::kVScales + (v_group * KEYS + v_step * kStep + 16 * i + 4 * v_quad) * 2) =
                u32x2{__builtin_amdgcn_perm(vpar[i][1], vpar[i][0], 0x05040100u),
                      __builtin_amdgcn_perm(vpar[i][3], vpar[i][2], 0x05040100u)};
        }
      }
    };

    f32x4 o[NT][G][MT], l[NT];
    float base[NT];
    float shrink[G];
#pragma unroll
    for (int g = 0; g < G; ++g) shrink[g] = 32768.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      base[n] = -INFINITY;
      l[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int y = 0; y < MT; ++y) o[n][g][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const uint32_t one2 = 0x3C003C00u;
    const u32x4 ones{one2, one2, one2, one2};

    // U steps from the c0-th of a round on
    auto compute = [&](const int (&key)[kPer], int holes, int c0, const uint8_t* buf) {
      // ---- scores: products of c - z, then the keys' scales
      f32x4 x[NT][2 * U];
#pragma unroll
      for (int u = 0; u < 2 * U; ++u)
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f32x4 acc[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = g * GROUP / 32; j < (g + 1) * GROUP / 32; ++j) {
            const u32x4 k = *reinterpret_cast<const u32x4*>(buf + ((2 * c0 + u) * kSteps + j) * 1024 + op_at(r, kb));
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] = mfma(k, qv[n][j], acc[n]);
          }
          const f32x4 sc = *reinterpret_cast<const f32x4*>(buf + L::kKScales + (g * KEYS + 32 * c0 + 16 * u + 4 * kb) * 4);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[n][u][i] = g == 0 ? acc[n][i] * sc[i] : fmaf(acc[n][i], sc[i], x[n][u][i]);
        }
      // ---- masks
      const int first = key[c0], end = key[c0 + U - 1] + kStep;
      const int miss = (holes >> (2 * c0)) & ((1 << (2 * U)) - 1);
      const bool whole = miss == 0 && end - first == U * kStep && end - 1 <= pos_lo &&
                         (a.window == 0 || first > pos_hi - a.window || end <= a.sinks);
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
          const bool here = !((miss >> u) & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = key[c0 + u / 2] + 16 * (u % 2) + 4 * kb + i;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const bool seen = here && t <= pos[n] && (a.window == 0 || t > pos[n] - a.window || t < a.sinks);
              x[n][u][i] = seen ? x[n][u][i] : -INFINITY;
            }
          }
        }
      }
      // ---- scales of the values, pairs of keys
      f16x2_t sv[G][4 * U];
      f16x2_t top2{0, 0};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        f16x2_t t{0, 0};
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(buf + L::kVScales + (g * KEYS + 32 * c0 + 16 * u + 4 * kb) * 2);
          const uint32_t v0 = v.x, v1 = v.y;
          sv[g][2 * u] = __builtin_bit_cast(f16x2_t, v0);
          sv[g][2 * u + 1] = __builtin_bit_cast(f16x2_t, v1);
          t = pk_max(t, pk_max(sv[g][2 * u], sv[g][2 * u + 1]));
        }
        top2 = pk_max(top2, t * pair16(shrink[g]));
      }
      // ---- running maximum and powers of two: one test for both
      bool grow = top2[0] > static_cast<_Float16>(1.0f) || top2[1] > static_cast<_Float16>(1.0f);
      float top[NT];
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
        grow |= t > base[n] + 15.0f;
      }
      if (__any(grow)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f16x2_t t{0, 0};
#pragma unroll
          for (int e = 0; e < 4 * U; ++e) t = pk_max(t, sv[g][e]);
          const float top = wave_max(fmaxf(static_cast<float>(t[0]), static_cast<float>(t[1])));
          const float next = fminf(shrink[g], __uint_as_float((251u - (__float_as_uint(top) >> 23)) << 23));
          const float f = next / shrink[g];
          shrink[g] = next;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= f;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float to = fmaxf(base[n], max_over_quads(top[n]) - 7.0f);
          const float fade = to == -INFINITY ? 1.0f : exp2_fast(base[n] - to);
          base[n] = to;
          l[n] *= fade;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= fade;
        }
      }
#pragma unroll
      for (int c = 0; c < U; ++c) {
        float p[NT][8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float from = base[n] == -INFINITY ? 0.0f : base[n];
          u32x4 pw;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f32x4& xs = x[n][2 * c + (e >> 1)];
            p[n][2 * e] = exp2_fast(xs[2 * (e & 1)] - from);
            p[n][2 * e + 1] = exp2_fast(xs[2 * (e & 1) + 1] - from);
            pw[e] = pack_pair<QMM_F16>(p[n][2 * e], p[n][2 * e + 1]);
          }
          l[n] = mfma(ones, pw, l[n]);
        }
        // ---- values
#pragma unroll
        for (int g = 0; g < G; ++g) {
          u32x4 pv[NT];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f16x2_t s2 = sv[g][4 * c + e] * pair16(shrink[g]);
#pragma unroll
            for (int n = 0; n < NT; ++n) pv[n][e] = weighted(p[n][2 * e], p[n][2 * e + 1], s2);
          }
#pragma unroll
          for (int y = 0; y < MT; ++y) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(
                buf + L::kVAt + ((c0 + c) * (D / 16) + g * MT + y) * L::kVStride + op_at(r, kb));
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][g][y] = mfma(v, pv[n], o[n][g][y]);
          }
        }
      }
    };

    // ---- rounds: this one's products, the next one's operands, the codes of
    // the one after, and the pages of the one after that
    Round now = round_of(0), next = round_of(1), then = round_of(2);
    if (rounds > 0) {
      fetch(now);
      if (now.key[kPer - 1] + kStep > sq.ctx) clean(now);
      expand(&lds[0][0]);
      if (rounds > 1) fetch(next);
    }
    __syncthreads();
    for (int round = 0; round < rounds; ++round) {
      if (round + 1 < rounds) {
        if (next.key[kPer - 1] + kStep > sq.ctx) clean(next);
        expand(&lds[(round + 1) & 1][0]);
      }
      if (round + 2 < rounds) fetch(then);
      const Round last = round_of(round + 3);
      const int holes = holes_of(now);
#pragma unroll
      for (int c = 0; c < kPer; c += U)
        if (now.key[c] != kBeyond) compute(now.key, holes, c, &lds[round & 1][0]);
      now = next;
      next = then;
      then = last;
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
      if (row >= rows) continue;
      const int tok = row / a.ratio;
      const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + kvh * a.ratio + row - tok * a.ratio;
      const float sum = l[n][0];
      const float inv = chunks > 1 ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float f = inv / shrink[g];
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

// Two blocks a compute unit where the registers allow it: one wavefront's
// products then run under the other's exponentials.
template <int DT, int D, int GROUP, int NT>
__global__ __launch_bounds__(256, NT * D <= 256 ? 2 : 1) void attention_chunk_kernel(AttnArgs a) {
  attention_chunk_block<DT, D, GROUP, NT>(a);
}

}  // namespace
}  // namespace qmm
