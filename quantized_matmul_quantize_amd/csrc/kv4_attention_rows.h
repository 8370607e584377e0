// kv4_attention_rows.h -- the attention kernel for a prefix that many rows see
// whole: the queries of all sequences of a group (products and their operand
// layouts: kv4_attention.h; here on 32 x 32 tiles).
//
// Every row sees every key, so there are no masks (but for keys whose page is
// none), and what a block expands serves eight wavefronts (four of D 256) of 32 rows each:
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
// Beside bf16 results that is little.  For binary16 ones what the rounding left, 5
// bits, is a second operand, and a value exact down to that step: with one of
// them 216 rows of 12 prefixes of 6000 tokens were 3.3e-4 off, 2.8e-4 with both.
// So nothing is left per score and group but one operation with the key's scale.
//
// Why so: two documents of 100000 tokens, 192 rows, D 128 in groups of 64.  Codes
// fetched a round ahead into registers left a round at memory's latency (3 us
// whatever D); straight to LDS six rounds ahead 257 -> 254 us.  Eight wavefronts in
// step met first at the matrix units and then at the vector units; with the
// second four a phase behind, and scales read before they are needed (returns
// in order made each wait one for all operands behind it), 254 -> 240 us.  Now a
// round of 64 keys takes ~2 us, of which two wavefronts' matrix instructions on a
// SIMD fill 0.85; the vector phase alone takes ~2100 cycles, ~330 operations that a
// wavefront alone issues no faster.  LDS is in use 33% of the time.
#pragma once

#include <utility>

#include "kv4_attention.h"
#include "kv4_deal.h"

namespace qmm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

template <int DT, int D, int GROUP>
struct Rows {
  static constexpr int kParts = DT == QMM_F16 ? 2 : 1;       // operands of a value
  static constexpr int kG = D / GROUP;
  static constexpr int kW = D == 256 ? 4 : 8;                // wavefronts: by the registers of sums and queries
  static constexpr int kThreads = kWave * kW;
  static constexpr int kStrip = 32;                          // rows of a wavefront
  static constexpr int kKeys = 8 * kW, kTiles = kKeys / 32;  // of a round
  static constexpr int kSteps = D / 16, kChannels = D / 32;
  // Operands of 1 KiB, [tile][k-extent] of keys, [tile][32 channels][16 keys] of
  // values (twice for two parts), each in two halves of 544 bytes: writers' eight lanes at a time then
  // meet every bank once, as readers' do.  Two buffers of each.
  static constexpr int kHalf = 544;
  static constexpr int kKOps = kTiles * kSteps * 2 * kHalf;
  static constexpr int kKBuffer = kKOps + kG * kKeys * 4;    // fp32 scales [group][key]
  static constexpr int kVPart = kTiles * kChannels * 2 * 2 * kHalf, kVBuffer = kParts * kVPart;
  // Codes as they lie in memory, kRing rounds: a round of few rows takes less
  // than memory does to answer.  Of each 16-key tile codes, then params [group][16].
  static constexpr int kCodes = 8 * D, kParams = 64 * kG;    // of a tile
  static constexpr int kRaw = kKeys / 16 * (kCodes + kParams);
  static constexpr int kSlot = 2 * kRaw;                     // keys, values
  static constexpr int kFit = (163840 - kW * kWave * 4 - 2 * (kKBuffer + kVBuffer)) / kSlot, kRing = kFit < 6 ? kFit : 6;
  static constexpr int kPagesAt = 2 * (kKBuffer + kVBuffer) + kRing * kSlot;      // a wavefront's next 64 pages
  static constexpr int kLds = kPagesAt + kW * kWave * 4;
  static constexpr int kLoads = kCodes / 1024 > 1 ? 3 : 2;   // of a wavefront a round
  // words of keys, and channels of a word of values, that a thread expands a round
  static constexpr int kWords = kKeys * D / 8 / kThreads;
  static_assert(kWords == D / 64, "two threads to every fourth word of a key");
};

// f(0), f(1), .. f(N - 1), their arguments constants
template <typename F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
  each(f, std::make_integer_sequence<int, N>{});
}

template <int DT, int D, int GROUP>
__device__ __forceinline__ void attention_rows_block(const SharedArgs& a, uint32_t id, uint8_t* lds) {
  using L = Rows<DT, D, GROUP>;
  constexpr int G = L::kG, KEYS = L::kKeys, T = L::kTiles, kSteps = L::kSteps, kCh = L::kChannels, kW = L::kW;
  constexpr int kWords = L::kWords, kGSteps = GROUP / 16;
  constexpr int kAhead = 4;                        // operands read before they are used
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r = lane & 31, h = lane >> 5;
  auto k_lds = [&](int i) { return lds + (i & 1) * L::kKBuffer; };
  auto v_lds = [&](int i) { return lds + 2 * L::kKBuffer + (i & 1) * L::kVBuffer; };
  uint8_t* const ring = lds + 2 * (L::kKBuffer + L::kVBuffer);

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
  if (split >= ch.chunks || sq.ctx == 0) return;
  const int key_lo = split * ch.chunk * kStep, key_hi = min(key_lo + ch.chunk * kStep, sq.ctx);
  const int rounds = (key_hi - key_lo + KEYS - 1) / KEYS;

  const int record = static_cast<int>(a.sh.record_bytes());
  const uint32_t page_bytes = static_cast<uint32_t>(a.sh.heads) * static_cast<uint32_t>(record);
  const uint32_t pages = static_cast<uint32_t>(a.sh.pages);
  const uint8_t* head = a.cache + static_cast<int64_t>(kvh) * record;
  const int32_t* table = a.table + item.table_row * a.table_stride;

  // What a thread expands of a round.  Keys: kWords of the words k_part + 4 i.
  // Values: of word v_word of two quads of tokens kWords of the even or the odd channels.
  const int k_part = lane & 3, k_side = lane >> 3 & 1;
  const int k_key = (lane >> 2 & 1) + (lane >> 4) * 2 + 8 * wave;
  const int k_from = k_key * (D / 2) + k_part * (D / 8) + k_side * (D / 16);
  constexpr int kPars = kWords * 32 > GROUP ? kWords * 32 / GROUP : 1;        // groups of a thread's words
  const int k_group = G > 1 ? k_side * kPars : 0;
  const int kp_from = KEYS / 16 * L::kCodes + (k_key >> 4) * L::kParams + k_group * 64 + (k_key & 15) * 4;
  const int k_to = (((k_key >> 5) * kSteps + 2 * k_side * kWords + (k_part >> 1)) * 2 + (k_part & 1)) * L::kHalf + (k_key & 31) * 16;
  const int v_part = lane & 1, v_half = lane >> 1 & 1, v_m = wave & 1, v_tile = D == 256 ? 0 : wave >> 1 & 1;
  const int v_word = D == 64 ? lane >> 2 & 7 : D == 128 ? lane >> 2 : (lane >> 2) + 16 * (wave >> 1);
  const int v_first = D == 64 ? (lane >> 5) + 2 * (wave >> 2) : D == 128 ? 2 * (wave >> 2) : 0;
  const int v_from = L::kRaw + (2 * v_tile + v_m) * L::kCodes + v_half * (2 * D) + 16 * v_word;
  const int vp_from = L::kRaw + KEYS / 16 * L::kCodes + (2 * v_tile + v_m) * L::kParams + v_word / (GROUP / 8) * 64 + 16 * v_half;
  // (rows 8 .. 15 and 24 .. 31 of an operand change places by fours: the banks of a word and the next differ)
  auto value_row = [](int row) { return row ^ ((row >> 3 & 1) << 2); };
  const int v_to = (((v_tile * kCh + v_word / 4) * 2 + v_m) * 2 + v_half) * L::kHalf;

  // The pages of 16-key tiles, one a lane, of 64 at a time, the next 64 on their
  // way to LDS: in order with the codes, so that nothing waits for them alone (and
  // every wait for LDS would wait for scalar loads).  A tile past the block's keys,
  // or whose page is not of this cache, is read through an empty resource: zeros.
  constexpr int kTiles16 = KEYS / 16, kBatch = kWave / kTiles16;              // rounds of a batch
  uint8_t* const my_pages = lds + L::kPagesAt + wave * kWave * 4;
  const uint32_t pages_to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(my_pages));
  const __amdgpu_buffer_rsrc_t table_rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<int32_t*>(table), 0, ((key_hi - 1) >> a.sh.shift) * 4 + 4, kBufferWord3);
  auto first_key = [&](int batch) { return key_lo + (batch * kWave + lane) * 16; };
  auto checked = [&](int page, int batch) { return first_key(batch) < key_hi && static_cast<uint32_t>(page) < pages ? page : -1; };
  auto pages_of = [&](int batch) {
    return checked(__builtin_amdgcn_raw_buffer_load_b32(table_rs, (first_key(batch) >> a.sh.shift) * 4, 0, 0), batch);
  };
  auto fetch_pages = [&](int batch) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(table_rs, (lds_ptr_t)(uintptr_t)pages_to, 4, (first_key(batch) >> a.sh.shift) * 4, 0,
                                             0, 0);
  };
  auto tile_of = [&](int page) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(head + static_cast<uint64_t>(static_cast<uint32_t>(max(page, 0))) * page_bytes), 0,
        page < 0 ? 0 : record, kBufferWord3);
  };
  // A wavefront loads the keys or the values of one 16-key tile of a round.
  const int l_tile = wave % kTiles16;
  const bool l_values = wave >= kTiles16;
  const int l_codes = (l_values ? a.sh.page * (D / 2) : 0) + 16 * lane;
  const int l_params = a.sh.page * (D + (l_values ? 4 * G : 0)) + (lane >> 2) * a.sh.page * 4 + 16 * (lane & 3);
  const int l_ahead = l_values ? 0 : 1;            // a deal: the values of a round, the keys of the next
  auto fetch = [&](int deal, const uint8_t* place_to, int page) {
    const int round = deal + l_ahead;
    const __amdgpu_buffer_rsrc_t rs = tile_of(page);
    const int place = (key_lo + round * KEYS + 16 * l_tile) & (a.sh.page - 1);
    const uint32_t to = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(place_to)) + (l_values ? L::kRaw : 0);
    if (D != 64 || lane < 32)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(to + l_tile * L::kCodes), 16, l_codes,
                                               place * (D / 2), 0, 0);
    if constexpr (D == 256)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(to + l_tile * L::kCodes + 1024), 16, l_codes + 1024,
                                               place * (D / 2), 0, 0);
    if (lane < 4 * G)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(to + kTiles16 * L::kCodes + l_tile * L::kParams), 16,
                                               l_params, place * 4, 0, 0);
  };

  const uint32_t magic = vgpr_const(Codes64::magic), magic_v = vgpr_const(0x44004400u);
  auto plus = [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, x) + __builtin_bit_cast(f16x2_t, y));
  };
  auto times = [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, x) * __builtin_bit_cast(f16x2_t, y));
  };
  float key_scale = 0.0f;
  // Expansions in pieces, to be put between matrix instructions; the first reads what the others need.
  constexpr int kPieces = kWords + 1;
  uint32_t kw[kWords], kp[kPars];
  auto expand_keys = [&](const uint8_t* raw, uint8_t* buf, int piece) {
    if (piece == 0) {
      if constexpr (kWords == 1) {
        kw[0] = *reinterpret_cast<const uint32_t*>(raw + k_from);
      } else if constexpr (kWords == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(raw + k_from);
        kw[0] = v.x;
        kw[1] = v.y;
      } else {
        const u32x4 v = *reinterpret_cast<const u32x4*>(raw + k_from);
#pragma unroll
        for (int w = 0; w < 4; ++w) kw[w] = v[w];
      }
#pragma unroll
      for (int i = 0; i < kPars; ++i) kp[i] = *reinterpret_cast<const uint32_t*>(raw + kp_from + 64 * i);
      return;
    }
    const int w = piece - 1;
    const uint32_t par = kp[w * kPars / kWords], z = 0xD400D400u + ((par >> 16) & 0xFu) * 0x00100010u;
    uint32_t p[4];
    Codes64::unpack(kw[w], magic, p);
    *reinterpret_cast<u32x4*>(buf + k_to + w * 4 * L::kHalf) = u32x4{plus(p[0], z), plus(p[1], z), plus(p[2], z), plus(p[3], z)};
    if (w * kPars % kWords == 0 && k_part == 0 && (G > 1 || k_side == 0))
      *reinterpret_cast<float*>(buf + L::kKOps + ((k_group + w * kPars / kWords) * KEYS + k_key) * 4) = kv4_scale(par) * key_scale;
  };
  uint32_t vz[4], vs[4], vw[4];
  auto expand_values = [&](const uint8_t* raw, uint8_t* buf, int piece) {
    if (piece == 0) {
      const uint32_t sel = v_part ? 0x07060302u : 0x05040100u;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const u32x4 codes = *reinterpret_cast<const u32x4*>(raw + v_from + 4 * D * q);
        const u32x4 par = *reinterpret_cast<const u32x4*>(raw + vp_from + 32 * q);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          vz[2 * q + e] = (__builtin_amdgcn_perm(par[2 * e + 1], par[2 * e], 0x0c060c02u) << 4 & 0x00F000F0u) | 0xC400C400u;   // -(4 + z / 16)
          vs[2 * q + e] = __builtin_amdgcn_perm(par[2 * e + 1], par[2 * e], 0x05040100u);
          // channel v_first at bit 4 of either token's half
          vw[2 * q + e] = __builtin_rotateright32(__builtin_amdgcn_perm(codes[2 * e + 1], codes[2 * e], sel), (4 * v_first + 28) & 31);
        }
      }
      return;
    }
    const int y = piece - 1;
    u32x4 v, rest;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t n = plus((__builtin_rotateright32(vw[e], 4 * y) & Codes64::mask) | magic_v, vz[e]);
      const uint32_t most = times(n, vs[e]);       // (a cast of v[e] in place would be one of v[0])
      v[e] = most;
      if constexpr (L::kParts == 2)
        rest[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, n), __builtin_bit_cast(f16x2_t, vs[e]),
                                                                         -__builtin_bit_cast(f16x2_t, most)));
    }
    const int row = 8 * (v_word & 3) + 2 * (v_first + y) + v_part;
    *reinterpret_cast<u32x4*>(buf + v_to + value_row(row) * 16) = v;
    if constexpr (L::kParts == 2) *reinterpret_cast<u32x4*>(buf + L::kVPart + v_to + value_row(row) * 16) = rest;
  };
  // Only LDS is shared, and the codes on their way are waited for in their turn.
  auto meet = [&] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  const int strips = (rows + L::kStrip - 1) / L::kStrip, tiles = (strips + kW - 1) / kW;
  // bf16 queries have one power of two a block, in which binary16 holds what lies
  // 2^31 below the largest.  The rows may be of several sequences, none of which
  // may cost another its bits: a tile takes its rows with a largest query below
  // `below` and down to 2^-12 of the largest of those (what is lost, 2^-27 of a row's
  // largest a channel, is less than its products' roundings), then those that are
  // left: none, but where a slot's queries are of another order, such as what an
  // unused one holds.
  float below = INFINITY;
  for (int tile = tile0; tile < tiles;) {
    // the strips are dealt evenly to the tiles
    const int strip = first_strip(tile, strips, tiles) + wave;
    const bool active = strip < first_strip(tile + 1, strips, tiles);
    const int row = strip * L::kStrip + r;
    bool live = active && row < rows;
    const int tok = live ? row / a.ratio : 0, qh = live ? kvh * a.ratio + row - tok * a.ratio : 0;
    const uint16_t* qp = a.q + (sq.row0 + tok) * a.q_ts + qh * a.q_hs + 8 * h;
    __syncthreads();                               // LDS is free: the rows before are done
    int now_pages = pages_of(0);                   // of the batch that is fetched
    u32x4 qv[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) qv[j] = live ? ld16(qp + 16 * j) : u32x4{0u, 0u, 0u, 0u};
    uint64_t there = __ballot(now_pages >= 0), there_next = 0;
    auto page_at = [&](int deal) { return __builtin_amdgcn_readlane(now_pages, (deal + l_ahead) % kBatch * kTiles16 + l_tile); };
    // The first round's keys go where the second's operands will be.
    if (!l_values) fetch(-1, k_lds(1), page_at(-1));
#pragma unroll
    for (int i = 0; i < L::kRing; ++i) fetch(i, ring + i * L::kSlot, page_at(i));
    fetch_pages(1);
    float unscale = 1.0f, left = 0.0f;             // left: rows below that are
    if constexpr (DT == QMM_BF16) {
      float* stat = reinterpret_cast<float*>(lds);
      float own = largest_bf16(qv, 0.0f);
      own = fmaxf(own, __shfl_xor(own, 32, kWave));
      float most = wave_max(own < below ? own : 0.0f), least = -wave_max(own > 0.0f ? -own : -INFINITY);
      if (lane == 0) {
        stat[wave] = most;
        stat[kW + wave] = least;
      }
      meet();
      most = stat[0];
      least = stat[kW];
#pragma unroll
      for (int w = 1; w < kW; ++w) {
        most = fmaxf(most, stat[w]);
        least = fminf(least, stat[kW + w]);
      }
      meet();
      const float floor = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(most * 0x1p-12f)));
      left = __any(least < floor) ? floor : 0.0f;
      // (rows without a finite query but 0 are of the first)
      if (own == 0.0f ? below < INFINITY : own < floor || own >= below) {
        live = false;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) qv[j] = u32x4{0u, 0u, 0u, 0u};
      }
      const QueryScale qs = query_scale(most);
      unscale = qs.up;
      to_f16(qv, qs.down);
    }
    key_scale = a.scale_log2 * unscale;
    wait_vm<L::kLoads * (L::kRing - 1) + 1>();     // the first keys and deal
    meet();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) expand_keys(k_lds(1), k_lds(0), i);
    for (int i = threadIdx.x; i < L::kVBuffer / 16; i += L::kThreads) reinterpret_cast<u32x4*>(v_lds(1))[i] = u32x4{0u, 0u, 0u, 0u};

    f32x16 o[kCh], x[T];
#pragma unroll
    for (int c = 0; c < kCh; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[c][i] = 0.0f;
    u32x4 p[T][2] = {};                              // nothing of the round before the first, whose values are zeros
    // p = 2^(x - base): at most 2^15, 2^7 where the maximum was last moved
    float base = -INFINITY, from = 0.0f, limit = -INFINITY, l = 0.0f;

    // The next deal but kRing, once all have read the one whose place it takes.
    int slot = 0;
    auto fetch_deal = [&](int deal) {
      const int mine = deal + l_ahead;
      if (mine % kBatch == 0) {
        now_pages = checked(*reinterpret_cast<const int*>(my_pages + 4 * lane), mine / kBatch);
        there_next = __ballot(now_pages >= 0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xc07f);        // read before its place is written
        fetch_pages(mine / kBatch + 1);
      }
      fetch(deal, ring + slot * L::kSlot, page_at(deal));
      slot = slot + 1 == L::kRing ? 0 : slot + 1;
    };
    // a deal's codes to operands
    auto expand = [&](int deal, int piece) {
      const uint8_t* raw = ring + slot * L::kSlot;
      if (piece % 2 == 0) expand_keys(raw, k_lds(deal + 1), piece / 2);
      else expand_values(raw, v_lds(deal), piece / 2);
    };

    // The matrix instructions of a round: the values of the round before, then
    // scores less the base they are taken at, products of a tile and group (a
    // unit) while the unit before is scaled.  Operands are read kAhead
    // instructions, scales a unit before their use: a wait for a read just sent
    // waits for all before it.
    constexpr bool kHalves = kW == 8;
    constexpr int kV = L::kParts * 2 * T * kCh, kN = kV + T * kSteps, kUnits = T * G;
    auto read_v = [&](const uint8_t* vb, int i) {
      const int c = i % kCh, m = i / kCh % (2 * T);           // m: 16 keys
      return *reinterpret_cast<const u32x4*>(vb + i / (2 * T * kCh) * L::kVPart +
                                             (((m / 2 * kCh + c) * 2 + m % 2) * 2 + h) * L::kHalf + value_row(r) * 16);
    };
    auto matrices = [&](int round) {
      const uint8_t* vb = v_lds(round + 1);
      const uint8_t* kb = k_lds(round);
      auto read = [&](int i) {
        return i < kV ? read_v(vb, i) : *reinterpret_cast<const u32x4*>(kb + ((i - kV) * 2 + h) * L::kHalf + 16 * r);
      };
      u32x4 ops[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ops[i] = read(i);
      f32x16 acc[2];
      f32x4 sc[4];
      auto scaled = [&](int unit, int c) {
        const int t = unit / G, grp = unit % G;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[t][4 * c + e] = fmaf(acc[unit % 2][4 * c + e], sc[c][e], grp == 0 ? -from : x[t][4 * c + e]);
      };
      __builtin_amdgcn_sched_barrier(0);
      each<kN>([&](auto index) {
        constexpr int i = index;
        const u32x4 op = ops[i % kAhead];
        if constexpr (i < kV) {
          o[i % kCh] = mfma32(op, p[i / kCh % (2 * T) / 2][i / kCh % 2], o[i % kCh]);
          if constexpr (i + kAhead < kN) ops[i % kAhead] = read(i + kAhead);
          if constexpr (!kHalves) {
            constexpr int first = i * 2 * kPieces / kV, last = (i + 1) * 2 * kPieces / kV;
            each<last - first>([&](auto k) { expand(round, first + k); });
          }
        } else {
          constexpr int j = (i - kV) % kSteps, unit = (i - kV) / kGSteps, at = j % kGSteps;
          if constexpr (at == 0)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[unit % 2][e] = 0.0f;
          acc[unit % 2] = mfma32(op, qv[j], acc[unit % 2]);
          constexpr int first = at * 4 / kGSteps, last = (at + 1) * 4 / kGSteps;
          each<last - first>([&](auto k) {
            constexpr int c = first + k;
            if constexpr (unit > 0) scaled(unit - 1, c);
            sc[c] = *reinterpret_cast<const f32x4*>(kb + L::kKOps + (unit % G * KEYS + 32 * (unit / G) + 8 * c + 4 * h) * 4);
          });
          if constexpr (i + kAhead < kN) ops[i % kAhead] = read(i + kAhead);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int c = 0; c < 4; ++c) scaled(kUnits - 1, c);
    };
    auto softmax = [&](int round) {
      // ---- keys of no page
      if (round % kBatch == 0 && round > 0) there = there_next;
      const int holes = static_cast<int>(~there >> (round % kBatch * kTiles16)) & ((1 << kTiles16) - 1);
      if (holes) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[t][e] = holes >> (2 * t + e / 8) & 1 ? -INFINITY : x[t][e];
      }
      // ---- running maximum
      float top = x[0][0];
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int e = 0; e < 16; e += 2) top = max3(top, x[t][e], x[t][e + 1]);
      if (__any(top > limit)) {
        const float both = fmaxf(top, __shfl_xor(top, 32, kWave));
        const float to = fmaxf(base, both + from - 7.0f);
        const float fade = to == -INFINITY ? 1.0f : exp2_fast(base - to);
        const float now_from = to == -INFINITY ? 0.0f : to, rest = unrounded(both, from, now_from, to > base);
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[t][e] = x[t][e] + (from - now_from) - rest;
#pragma unroll
        for (int c = 0; c < kCh; ++c) o[c] *= fade;
        l *= fade;
        base = to;
        from = now_from;
        limit = to == -INFINITY ? -INFINITY : 15.0f;
      }
      // ---- probabilities and sums
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p0 = exp2_fast(x[t][2 * i]), p1 = exp2_fast(x[t][2 * i + 1]);
          l += p0 + p1;
          p[t][i / 4][i % 4] = pack_pair<QMM_F16>(p0, p1);
        }
    };

    // A round is a phase of matrix instructions and one of vector work: the softmax
    // and the expansion of a deal.  The second four wavefronts, which share the
    // SIMDs with the first four, are a phase behind, so that the one's matrix
    // instructions run under the other's vector work.  Deal i is expanded in phase
    // 2 i by the second half and 2 i + 1 by the first, and used from phase 2 i + 2
    // on, when its place in the ring is filled again.  (Four wavefronts have a SIMD
    // each and expand between matrix instructions.)
    const bool second = kHalves && wave >= 4;
    // (the first two pieces read the codes)
    auto expand_rest = [&](int deal) { each<2 * kPieces - 2>([&](auto k) { expand(deal, k + 2); }); };
    meet();
    if (second) {
      expand(0, 0), expand(0, 1);
      expand_rest(0);
      meet();
    }
    for (int round = 0; round < rounds; ++round) {
      if (!second && round > 0) fetch_deal(round - 1 + L::kRing);
      if (active) {
        __builtin_amdgcn_s_setprio(1);
        matrices(round);
        __builtin_amdgcn_s_setprio(0);
      } else if constexpr (!kHalves) {
        expand(round, 0), expand(round, 1);
        expand_rest(round);
      }
      if constexpr (kHalves) {
        if (second) wait_vm<L::kLoads * (L::kRing - 2)>();
        meet();
        if (second) fetch_deal(round + L::kRing);
        const int deal = second ? round + 1 : round;
        expand(deal, 0), expand(deal, 1);
        __builtin_amdgcn_sched_barrier(0);
        if (active) softmax(round);
        expand_rest(deal);
        if (second && round + 1 == rounds) break;
      } else if (active) {
        softmax(round);
      }
      if (!second) wait_vm<L::kLoads * (L::kRing - 2)>();
      meet();
    }
    if (active) {
      const uint8_t* vb = v_lds(rounds - 1);
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        o[i % kCh] = mfma32(read_v(vb, i), p[i / kCh % (2 * T) / 2][i / kCh % 2], o[i % kCh]);
      }
    }

    wait_vm<0>();                                  // nothing is on its way to LDS any more
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
    below = left > 0.0f ? left : INFINITY;
    tile += left > 0.0f ? 0 : a.p_row_tiles;
  }
}

template <int DT, int D, int GROUP>
__global__ __launch_bounds__((Rows<DT, D, GROUP>::kThreads), (Rows<DT, D, GROUP>::kW / 4)) void attention_rows_kernel(SharedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[Rows<DT, D, GROUP>::kLds];
  attention_rows_block<DT, D, GROUP>(a, blockIdx.x, lds);
}

}  // namespace
}  // namespace qmm
