// kv4_attention_rows.h -- the attention kernel for a prefix that many rows see
// whole: the queries of all sequences of a group (products and their operand
// layouts: kv4_attention.h; here on 32 x 32 tiles).
//
// Every row sees every key, so there are no masks (but for keys whose page is
// none), and what a block expands serves four wavefronts of 32 rows each:
//
//   S^T = K Q^T   32 keys x 16 channels first, codes less their zero-points
//                 (exact in binary16), q second; a lane ends with 16 keys of
//                 one row, scaled by the keys' scales in fp32;
//   O^T += V^T P^T  32 channels x 16 keys first, the lane's own probabilities
//                 second (the order of the keys in an operand is that in which
//                 the first product leaves them).
//
// Values are expanded with their scales: (c - z) / 16 is exact, its product with
// the scale is rounded to binary16 (2^-11; below 2^-14 a step of 2^-24, 2^-20 of
// a value), and no scale overflows; probabilities are rounded once to binary16.
// So nothing is left per score and group but one operation with the key's scale.
#pragma once

#include "kv4_attention.h"

namespace qmm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <int D, int GROUP>
struct Rows {
  static constexpr int kG = D / GROUP;
  static constexpr int kStrip = 32;                          // rows of a wavefront
  static constexpr int kKeys = D == 256 ? 32 : 64;           // of a round
  static constexpr int kTiles = kKeys / 32, kSteps = D / 16, kChannels = D / 32;
  // Operands of 1 KiB, [tile][k-extent] of keys, [tile][32 channels][16 keys] of
  // values, each in two halves of 544 bytes: writers' eight lanes at a time then
  // meet every bank once, as readers' do.
  static constexpr int kHalf = 544;
  static constexpr int kKOps = kTiles * kSteps * 2 * kHalf;
  static constexpr int kKBuffer = kKOps + kG * kKeys * 4;    // fp32 scales [group][key]
  static constexpr int kVBuffer = kTiles * kChannels * 2 * 2 * kHalf;
  static constexpr int kLds = 2 * (kKBuffer + kVBuffer);
  static constexpr int kWords = kKeys * D / 8 / 256;         // of keys, that a thread expands
  static constexpr int kNibbles = D == 64 ? 2 : 4;           // channels of values
};

// Blocks a compute unit: by the registers of the sums (D / 32 x 16) and queries.
constexpr int rows_occupancy(int D) { return D < 256 ? 2 : 1; }

template <int DT, int D, int GROUP>
__device__ __forceinline__ void attention_rows_block(const SharedArgs& a, uint32_t id, uint8_t* lds) {
  using L = Rows<D, GROUP>;
  constexpr int G = L::kG, KEYS = L::kKeys, kTiles = L::kTiles, kSteps = L::kSteps, kCh = L::kChannels;
  constexpr int kGSteps = GROUP / 16, kPages = KEYS / 16;
  constexpr int kAhead = 4;                        // operands read before they are used
  constexpr int kAluMayCross = 0x6;                // sched_barrier: scalar and vector arithmetic
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r = lane & 31, h = lane >> 5;
  auto k_lds = [&](int i) { return lds + (i & 1) * L::kKBuffer; };
  auto v_lds = [&](int i) { return lds + 2 * L::kKBuffer + (i & 1) * L::kVBuffer; };

  // row tiles of the same keys eight blocks apart: on one die, whose cache holds the codes
  const uint32_t eight = id % 8;
  id /= 8;
  const int tile0 = static_cast<int>(id % a.p_row_tiles);
  id = id / a.p_row_tiles * 8 + eight;
  const int kvh = static_cast<int>(id % a.sh.heads);
  id /= a.sh.heads;
  const int split = static_cast<int>(id % a.p_splits);
  const int g = static_cast<int>(id / a.p_splits);
  if (g >= a.n_groups) return;
  const Item item = prefix_item(a, g);
  const Sequence sq = item.sq;
  const int rows = sq.n * a.ratio;
  const Chunks ch = part_chunks<kPrefix>(a, item);
  if (split >= ch.chunks) return;
  const int key_lo = split * ch.chunk * kStep, key_hi = min(key_lo + ch.chunk * kStep, sq.ctx);
  const int rounds = (key_hi - key_lo + KEYS - 1) / KEYS;

  const int record = static_cast<int>(a.sh.record_bytes());
  const uint32_t page_bytes = static_cast<uint32_t>(a.sh.heads) * static_cast<uint32_t>(record);
  const uint32_t pages = static_cast<uint32_t>(a.sh.pages);
  const uint8_t* head = a.cache + static_cast<int64_t>(kvh) * record;
  typedef const __attribute__((address_space(4))) int32_t* table_t;
  const table_t table = (table_t)(a.table + item.table_row * a.table_stride);

  // What a thread expands of a round.  Keys: kWords words (every fourth of the
  // key) from one piece of its row.  Values: of word v_word of two quads of
  // tokens the even or the odd channels.
  const int k_tile = D == 256 ? wave >> 1 : wave;             // of 16 keys
  const int k_key = D == 256 ? (lane >> 2 & 7) + 8 * (wave & 1) : lane >> 2;
  const int k_part = lane & 3, k_first = D == 256 ? 4 * (lane >> 5) : 0;
  const int k_at = k_key * (D / 2) + k_part * (D / 8) + 4 * k_first, kp_at = a.sh.page * D + 4 * k_key;
  const int k_to = ((k_tile / 2 * kSteps + 2 * k_first + (k_part >> 1)) * 2 + (k_part & 1)) * L::kHalf +
                   (16 * (k_tile & 1) + k_key) * 16;
  const int v_part = lane & 1, v_half = lane >> 1 & 1;
  const int v_word = D == 64 ? lane >> 2 & 7 : D == 128 ? lane >> 2 : (lane >> 2) + 16 * (wave >> 1);
  const int v_first = D == 64 ? 2 * (lane >> 5) : 0;          // of its nibbles
  const int v_m = wave & 1, v_tile = D == 256 ? 0 : wave >> 1;
  const int v_group = v_word / (GROUP / 8);
  const int v_at = a.sh.page * (D / 2) + v_half * (2 * D) + 16 * v_word;
  const int vp_at = a.sh.page * (D + 4 * G) + v_group * a.sh.page * 4 + 16 * v_half;
  // (rows 8 .. 15 and 24 .. 31 of an operand lie four rows apart from their order: see value_row)
  auto value_row = [](int row) { return row ^ ((row >> 3 & 1) << 2); };
  const int v_to = (((v_tile * kCh + v_word / 4) * 2 + v_m) * 2 + v_half) * L::kHalf;

  // A 16-key tile past the block's keys, or whose page is not of this cache, is
  // read through an empty resource: zeros.
  auto page_at = [&](int key) {
    const int page = table[max(min(key, sq.ctx - 1), 0) >> a.sh.shift];
    return key < key_hi ? page : -1;
  };
  auto tile_of = [&](int page) {
    const bool here = static_cast<uint32_t>(page) < pages;
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(head + static_cast<uint64_t>(static_cast<uint32_t>(here ? page : 0)) * page_bytes), 0,
        here ? record : 0, kBufferWord3);
  };
  uint32_t k_raw[L::kWords], k_par[G];
  u32x4 v_raw[2], v_par[2];
  auto fetch = [&](int round, int k_page, int v_page) {
    const int key = key_lo + round * KEYS;
    {
      const __amdgpu_buffer_rsrc_t rs = tile_of(k_page);
      const int place = (key + 16 * k_tile) & (a.sh.page - 1);
      if constexpr (L::kWords == 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, k_at, place * (D / 2), 0));
        k_raw[0] = v.x;
        k_raw[1] = v.y;
      } else {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, k_at, place * (D / 2), 0));
#pragma unroll
        for (int w = 0; w < 4; ++w) k_raw[w] = v[w];
      }
#pragma unroll
      for (int i = 0; i < G; ++i)
        k_par[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, kp_at + i * a.sh.page * 4, place * 4, 0);
    }
    {
      const __amdgpu_buffer_rsrc_t rs = tile_of(v_page);
      const int place = (key + 32 * v_tile + 16 * v_m) & (a.sh.page - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v_raw[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, v_at + i * 4 * D, place * (D / 2), 0));
        v_par[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, vp_at + 32 * i, place * 4, 0));
      }
    }
  };
  auto k_page_of = [&](int round) { return page_at(key_lo + round * KEYS + 16 * k_tile); };
  auto v_page_of = [&](int round) { return page_at(key_lo + round * KEYS + 32 * v_tile + 16 * v_m); };

  const uint32_t magic = vgpr_const(Codes64::magic), magic_v = vgpr_const(0x44004400u);
  auto plus = [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, x) + __builtin_bit_cast(f16x2_t, y));
  };
  auto times = [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, x) * __builtin_bit_cast(f16x2_t, y));
  };
  float key_scale = 0.0f;
  auto expand_keys = [&](uint8_t* buf) {
#pragma unroll
    for (int w = 0; w < L::kWords; ++w) {
      // word k_part + 4 (k_first + w), in the 32 channels k_first + w
      uint32_t par = k_par[0];
#pragma unroll
      for (int i = 1; i < G; ++i) par = (k_first + w) / (GROUP / 32) == i ? k_par[i] : par;
      const uint32_t z = 0xD400D400u + ((par >> 16) & 0xFu) * 0x00100010u;
      uint32_t p[4];
      Codes64::unpack(k_raw[w], magic, p);
      *reinterpret_cast<u32x4*>(buf + k_to + w * 4 * L::kHalf) = u32x4{plus(p[0], z), plus(p[1], z), plus(p[2], z), plus(p[3], z)};
    }
    if (k_part == 0 && k_first == 0) {
#pragma unroll
      for (int i = 0; i < G; ++i)
        *reinterpret_cast<float*>(buf + L::kKOps + (i * KEYS + 16 * k_tile + k_key) * 4) = kv4_scale(k_par[i]) * key_scale;
    }
  };
  auto expand_values = [&](uint8_t* buf) {
    uint32_t z[4], s[4], w[4];
    const uint32_t sel = v_part ? 0x07060302u : 0x05040100u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t p0 = v_par[e >> 1][2 * (e & 1)], p1 = v_par[e >> 1][2 * (e & 1) + 1];
      z[e] = (__builtin_amdgcn_perm(p1, p0, 0x0c060c02u) << 4 & 0x00F000F0u) | 0xC400C400u;      // -(4 + z / 16)
      s[e] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
      w[e] = __builtin_amdgcn_perm(v_raw[e >> 1][2 * (e & 1) + 1], v_raw[e >> 1][2 * (e & 1)], sel) >> (4 * v_first);
    }
#pragma unroll
    for (int y = 0; y < L::kNibbles; ++y) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = times(plus(((y == 0 ? w[e] << 4 : w[e] >> (4 * y - 4)) & Codes64::mask) | magic_v, z[e]), s[e]);
      const int row = 8 * (v_word & 3) + 2 * (v_first + y) + v_part;
      *reinterpret_cast<u32x4*>(buf + v_to + value_row(row) * 16) = v;
    }
  };

  const int strips = (rows + L::kStrip - 1) / L::kStrip, tiles = (strips + kWaves - 1) / kWaves;
  for (int tile = tile0; tile < tiles; tile += a.p_row_tiles) {
    // the strips are dealt evenly to the tiles
    const int strip = tile * strips / tiles + wave;
    const bool active = strip < (tile + 1) * strips / tiles;
    const int row = strip * L::kStrip + r;
    const bool live = active && row < rows;
    const int tok = live ? row / a.ratio : 0, qh = live ? kvh * a.ratio + row - tok * a.ratio : 0;
    const uint16_t* qp = a.q + (sq.row0 + tok) * a.q_ts + qh * a.q_hs + 8 * h;
    fetch(0, k_page_of(0), v_page_of(0));
    u32x4 qv[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) qv[j] = live ? ld16(qp + 16 * j) : u32x4{0u, 0u, 0u, 0u};
    float unscale = 1.0f;
    __syncthreads();                               // LDS is free: the rows before are done
    if constexpr (DT == QMM_BF16) {
      float* stat = reinterpret_cast<float*>(lds);
      float most = wave_max(largest_bf16(qv, 0.0f));
      if (lane == 0) stat[wave] = most;
      __syncthreads();
      most = fmaxf(fmaxf(stat[0], stat[1]), fmaxf(stat[2], stat[3]));
      const QueryScale qs = query_scale(most);
      __syncthreads();
      unscale = qs.up;
      to_f16(qv, qs.down);
    }
    key_scale = a.scale_log2 * unscale;
    expand_keys(k_lds(0));
    expand_values(v_lds(0));
    if (rounds > 1) fetch(1, k_page_of(1), v_page_of(1));

    f32x16 o[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
    // p = 2^(x - base): at most 2^15, 2^7 where the maximum was last moved
    float base = -INFINITY, from = 0.0f, limit = -INFINITY, l = 0.0f;
    int k_page = k_page_of(2), v_page = v_page_of(2);
    __syncthreads();

    for (int round = 0; round < rounds; ++round) {
      const uint8_t* kb = k_lds(round);
      const uint8_t* vb = v_lds(round);
      const int k_after = k_page_of(round + 3), v_after = v_page_of(round + 3);
      if (active) {
        // ---- scores less the base they are taken at
        f32x16 x[kTiles], acc[kTiles];
        {
          constexpr int kOps = kSteps * kTiles;
          u32x4 k[kAhead];
          auto read = [&](int i) {
            return *reinterpret_cast<const u32x4*>(kb + ((i % kTiles * kSteps + i / kTiles) * 2 + h) * L::kHalf + 16 * r);
          };
#pragma unroll
          for (int i = 0; i < kAhead; ++i) k[i] = read(i);
          __builtin_amdgcn_sched_barrier(kAluMayCross);
#pragma unroll
          for (int i = 0; i < kOps; ++i) {
            const int t = i % kTiles, j = i / kTiles, grp = j / kGSteps;
            if (j % kGSteps == 0)
#pragma unroll
              for (int e = 0; e < 16; ++e) acc[t][e] = 0.0f;
            acc[t] = mfma32(k[i % kAhead], qv[j], acc[t]);
            if (i + kAhead < kOps) k[i % kAhead] = read(i + kAhead);
            __builtin_amdgcn_sched_barrier(kAluMayCross);
            if (j % kGSteps == kGSteps - 1)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const f32x4 sc = *reinterpret_cast<const f32x4*>(kb + L::kKOps + (grp * KEYS + 32 * t + 8 * c + 4 * h) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  x[t][4 * c + e] = fmaf(acc[t][4 * c + e], sc[e], grp == 0 ? -from : x[t][4 * c + e]);
              }
          }
        }
        // ---- keys of no page
        int holes = 0;
#pragma unroll
        for (int t = 0; t < kPages; ++t)
          holes |= static_cast<uint32_t>(page_at(key_lo + round * KEYS + 16 * t)) < pages ? 0 : 1 << t;
        if (holes) {
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[t][e] = holes >> (2 * t + e / 8) & 1 ? -INFINITY : x[t][e];
        }
        // ---- running maximum
        float top = x[0][0];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 16; e += 2) top = max3(top, x[t][e], x[t][e + 1]);
        if (__any(top > limit)) {
          const float both = fmaxf(top, __shfl_xor(top, 32, kWave));
          const float to = fmaxf(base, both + from - 7.0f);
          const float fade = to == -INFINITY ? 1.0f : exp2_fast(base - to);
          const float now_from = to == -INFINITY ? 0.0f : to;
#pragma unroll
          for (int t = 0; t < kTiles; ++t) x[t] += from - now_from;
#pragma unroll
          for (int c = 0; c < kCh; ++c) o[c] *= fade;
          l *= fade;
          base = to;
          from = now_from;
          limit = to == -INFINITY ? -INFINITY : 15.0f;
        }
        // ---- probabilities
        u32x4 p[kTiles][2];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float p0 = exp2_fast(x[t][e]), p1 = exp2_fast(x[t][e + 1]);
            l += p0 + p1;
            p[t][e / 8][e / 2 % 4] = pack_pair<QMM_F16>(p0, p1);
          }
        // ---- sums
        {
          constexpr int kOps = kTiles * 2 * kCh;
          u32x4 v[kAhead];
          auto read = [&](int i) {
            const int c = i % kCh, m = i / kCh;               // m: 16 keys
            return *reinterpret_cast<const u32x4*>(vb + (((m / 2 * kCh + c) * 2 + m % 2) * 2 + h) * L::kHalf + value_row(r) * 16);
          };
#pragma unroll
          for (int i = 0; i < kAhead; ++i) v[i] = read(i);
          __builtin_amdgcn_sched_barrier(kAluMayCross);
#pragma unroll
          for (int i = 0; i < kOps; ++i) {
            const int c = i % kCh, m = i / kCh;
            o[c] = mfma32(v[i % kAhead], p[m / 2][m % 2], o[c]);
            if (i + kAhead < kOps) v[i % kAhead] = read(i + kAhead);
            __builtin_amdgcn_sched_barrier(kAluMayCross);
          }
        }
      }
      if (round + 1 < rounds) {
        expand_keys(k_lds(round + 1));
        expand_values(v_lds(round + 1));
        if (round + 2 < rounds) fetch(round + 2, k_page, v_page);
      }
      k_page = k_after;
      v_page = v_after;
      // only LDS is shared: the codes on their way need not have come
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    }

    // ---- results: row r, channels 8 c + 4 h of every 32
    l += __shfl_xor(l, 32, kWave);
    if (live) {
      const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + qh;
      const int64_t at = slot_of<kPrefix>(a, rh, split);
#pragma unroll
      for (int c = 0; c < kCh; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(a.part_o + at * D + 32 * c + 8 * i + 4 * h) =
              f32x4{o[c][4 * i], o[c][4 * i + 1], o[c][4 * i + 2], o[c][4 * i + 3]} * 16.0f;
      if (h == 0) a.part_ml[at] = make_float2(base, l);
    }
  }
}

template <int DT, int D, int GROUP>
__global__ __launch_bounds__(256, rows_occupancy(D)) void attention_rows_kernel(SharedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Rows<D, GROUP>::kLds];
  attention_rows_block<DT, D, GROUP>(a, blockIdx.x, lds);
}

}  // namespace
}  // namespace qmm
