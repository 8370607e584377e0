// kv4_attention.hip -- causal attention over the 4-bit paged cache (the
// format and the masks are stated in include/qmm.h).
//
// One kernel serves decode and chunks.  The rows of one sequence and kv head
// (its queries times the query heads that share the kv head) are taken 16 NT
// at a time, the keys 32 at a time, in one pass with a running maximum and sum:
//
//   S^T = K Q^T   codes of 16 keys x 32 channels as the first operand, 16 rows
//                 of q as the second, so a lane ends with 4 keys of one row;
//   O^T += V^T P^T  codes of 16 channels x 32 keys first, the same lane's
//                 probabilities second: the lane that computed S^T[4 kb + i][r]
//                 of two 16-key tiles holds exactly the eight k-entries that
//                 the second product wants of it, so the probabilities never
//                 leave their lane, and the running statistics of row r belong
//                 to the lanes that hold column r of O^T.
//
// The codes enter the matrix cores as they are, as the 16-bit floats 128 + c
// (16 + c where q is binary16), exactly; offset, zero-point and scale are
// applied around the products:
//   x[t] = sum_g s[t,g] ((sum_{d in g} q_d (off + c)) - (off + z[t,g]) sum_{d in g} q_d)
//   o[d] = 2^e[g] (sum_t p'[t] (16 + c) - sum_t p'[t] (16 + z[t,g])),  p' = p s[t,g] 2^-e[g]
// with the second sum of o one more product whose first operand is 16 + z.
// p and p' are rounded to binary16 (2^-12 each; both sums see the same p'), for
// either type of q: bf16 would cost 2^-9.  Its range is kept by the two powers
// of two that are moved only when they must be: p lies below 2^15 (and reaches
// 2^7 where the maximum was last moved, so that what is lost below 2^-25 is
// 2^-32 of the largest), s 2^-e below 1.  The scores, maxima and sums of p
// stay in fp32.

#include <algorithm>

#include "kv4_device.h"

namespace qmm {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kStep = 32;            // keys per step: one k-extent of the second product

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

template <int DT>
__device__ __forceinline__ f32x4 mfma_q(const uint32_t a[4], u32x4 b, f32x4 c) {
  const u32x4 av{a[0], a[1], a[2], a[3]};
  if constexpr (DT == QMM_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, av), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
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
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int D, int GROUP>
struct Tile {
  static constexpr int kG = D / GROUP;
  static constexpr int kCodeLoads = D / 64;                 // 1 KiB loads of a 16-key tile's codes
  static constexpr int kLoads = 2 * (kCodeLoads + 1);       // of a step
  static constexpr int kBytes = 16 * D + 128 * kG;          // K codes, V codes, K params, V params
  static constexpr int kStepBytes = 2 * kBytes;
  static constexpr int kChunks = D / 32;                    // 16-byte pieces of a key's codes
  static constexpr int kMTiles = GROUP / 16;                // channel tiles of a group
  // Rotation of a key's pieces within its row in LDS: the 16 lanes that read
  // one piece of 16 keys then meet every bank once.
  static __device__ __forceinline__ int rot(int r) { return r * kChunks / 16; }
};

template <int DT, int D, int GROUP, int NT, bool WS>
__device__ __forceinline__ void attention_block(const AttnArgs& a) {
  using L = Tile<D, GROUP>;
  constexpr int G = L::kG, kSteps = D / 32, kStages = 3;
  constexpr int MT = L::kMTiles;
  constexpr int kRows = 16 * NT * (WS ? 1 : kWaves);
  constexpr float kOff = Int4Magic<DT>::offset;
  __shared__ __attribute__((aligned(16))) uint8_t ring[kWaves][kStages][L::kStepBytes];

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int r = lane & 15, kb = lane >> 4;

  int64_t id = blockIdx.x;
  const int split = static_cast<int>(id % a.splits);
  id /= a.splits;
  const int kvh = static_cast<int>(id % a.sh.heads);
  id /= a.sh.heads;
  const int tile0 = static_cast<int>(id % a.row_tiles);
  const int b = static_cast<int>(id / a.row_tiles);
  const Sequence sq = sequence_of(a, b);
  const int rows = sq.n * a.ratio;

  // byte offsets of this lane's loads in a record, without the tile's place
  int voff[L::kCodeLoads];
#pragma unroll
  for (int n = 0; n < L::kCodeLoads; ++n) {
    const int p = 64 * n + lane, R = p / L::kChunks;
    voff[n] = p < D / 2 ? R * (D / 2) + 16 * ((p - L::rot(R)) & (L::kChunks - 1)) : a.sh.page * (D / 2) + 16 * (p - D / 2);
  }
  const int poff = a.sh.page * D + (lane / 4) * a.sh.page * 4 + 16 * (lane & 3);   // [K, V][group][page] words
  const int64_t record = a.sh.record_bytes();
  const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(&ring[wave][0][0]));
  const __attribute__((address_space(4))) int32_t* table =
      (const __attribute__((address_space(4))) int32_t*)(a.table + b * a.table_stride);

  // The pages of the two 16-key tiles from key t0 (-1 past the context).
  struct Pages {
    int p[2];
  };
  auto pages_of = [&](int t0) {
    Pages x;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + 16 * u;
      x.p[u] = t < sq.ctx ? table[t >> a.sh.shift] : -1;
    }
    return x;
  };
  int holes = 0;     // bit 2 stage + u: that tile has no page of this cache
  // Requests the 32 keys from key t0 into a stage.  A 16-key tile past the
  // context, or whose page is not of this cache, is read through an empty
  // resource: zeros, so scales of 0.
  auto issue = [&](int t0, Pages pages, int stage) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int t = t0 + 16 * u;
      const int64_t page = pages.p[u];
      const bool here = page >= 0 && page < a.sh.pages;
      holes = (holes & ~(1 << (2 * stage + u))) | (here ? 0 : 1 << (2 * stage + u));
      const uint8_t* rec = a.cache + (here ? (page * a.sh.heads + kvh) * record : 0);
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(rec), 0, here ? static_cast<int>(record) : 0, kBufferWord3);
      const int place = t & (a.sh.page - 1);
      const uint32_t dst = ring0 + stage * L::kStepBytes + u * L::kBytes;
#pragma unroll
      for (int n = 0; n < L::kCodeLoads; ++n)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(dst + n * 1024), 16, voff[n],
                                                 place * (D / 2), 0, 0);
      if (lane < 8 * G)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(uintptr_t)(dst + 16 * D), 16, poff, place * 4, 0, 0);
    }
  };

  for (int tile = tile0; tile * kRows < rows || tile == 0; tile += a.row_tiles) {
    if (rows == 0) break;
    const int row_lo = tile * kRows + (WS ? 0 : wave * 16 * NT);          // this wavefront's rows
    const int row_hi = min(row_lo + 16 * NT, rows) - 1;
    const int tok_lo = row_lo / a.ratio, tok_hi = (row_hi < row_lo ? row_lo : row_hi) / a.ratio;
    const int pos_lo = sq.first + tok_lo, pos_hi = row_hi < row_lo ? -1 : sq.first + tok_hi;
    // the block's steps: every wavefront splits the same range into chunks
    const int blk_lo = sq.first + tile * kRows / a.ratio;
    const int blk_hi = sq.first + (min(tile * kRows + kRows, rows) - 1) / a.ratio;
    const Steps st = steps_of(a, blk_lo, blk_hi);
    const int chunks = max(1, (st.count + a.chunk - 1) / a.chunk);
    if (split >= chunks) continue;
    const int s_lo = split * a.chunk + (WS ? wave : 0), s_hi = min(split * a.chunk + a.chunk, st.count);
    constexpr int kStride = WS ? kWaves : 1;

    // queries as second operands, their sums per group, and their positions
    u32x4 qv[NT][kSteps];
    float qsum[NT][G];
    int pos[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row_lo + 16 * n + r;
      const bool live = row < rows;
      const int tok = live ? row / a.ratio : 0, head = live ? kvh * a.ratio + row - tok * a.ratio : 0;
      pos[n] = live ? sq.first + tok : -1;
      const uint16_t* qp = a.q + (sq.row0 + tok) * a.q_ts + head * a.q_hs + 8 * kb;
#pragma unroll
      for (int j = 0; j < kSteps; ++j) qv[n][j] = live ? ld16(qp + 32 * j) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float s = 0.0f;
#pragma unroll
        for (int j = g * GROUP / 32; j < (g + 1) * GROUP / 32; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            s += DT == QMM_BF16 ? bf16lo_to_f32(qv[n][j][w]) + bf16hi_to_f32(qv[n][j][w])
                                : f16lo_to_f32(qv[n][j][w]) + f16hi_to_f32(qv[n][j][w]);
        qsum[n][g] = sum_over_quads(s);
      }
    }

    f32x4 o[NT][G][MT], corr[NT][G];
    // p = 2^(x - base); base -inf until a key is seen, then at least 2^-15
    // below and at most 2^7 above the largest x
    float base[NT], l[NT];
    float shrink[G];        // 2^-e[g], the same in every lane
#pragma unroll
    for (int g = 0; g < G; ++g) shrink[g] = 32768.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      base[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        corr[n][g] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < MT; ++x) o[n][g][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
    const uint32_t magic_q = vgpr_const(Int4Magic<DT>::kMagic);
    const uint32_t magic_v = vgpr_const(Int4Magic<QMM_F16>::kMagic);
    constexpr uint32_t kNibbles = 0x03C003C0u;

    auto compute = [&](int t0, int stage) {
      const uint8_t* slot = &ring[wave][stage][0];
      // ---- scores
      f32x4 x[NT][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t* kp = slot + u * L::kBytes;
        uint32_t w[kSteps];
        if constexpr (D == 64) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(kp + 16 * (2 * r + (((kb >> 1) + L::rot(r)) & 1)) + 8 * (kb & 1));
          w[0] = v.x; w[1] = v.y;
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
        f32x4 acc[NT];
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float c = -kOff * qsum[n][g];
            acc[n] = f32x4{c, c, c, c};
          }
#pragma unroll
          for (int j = g * GROUP / 32; j < (g + 1) * GROUP / 32; ++j) {
            uint32_t av[4];
            Int4Magic<DT>::unpack(w[j], magic_q, av);
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n] = mfma_q<DT>(av, qv[n][j], acc[n]);
          }
          u32x4 par = *reinterpret_cast<const u32x4*>(kp + 16 * D + g * 64 + 16 * kb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = kv4_scale(par[i]), z = kv4_zero(par[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float v = s * fmaf(-z, qsum[n][g], acc[n][i]);
              x[n][u][i] = g == 0 ? v : x[n][u][i] + v;
            }
          }
        }
      }
      // ---- masks: only steps that some row does not see whole (columns past
      // the rows hold zeros of q: finite, and never stored)
      const bool whole = t0 + kStep - 1 <= pos_lo && (a.window == 0 || t0 > pos_hi - a.window || t0 + kStep <= a.sinks);
      bool stored[8];      // memory past the context may hold anything
#pragma unroll
      for (int e = 0; e < 8; ++e) stored[e] = true;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) x[n][u] *= a.scale_log2;
      const int missing = (holes >> (2 * stage)) & 3;
      if (!whole || missing) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tt = t0 + 16 * u;
          const bool here = !((missing >> u) & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = tt + 4 * kb + i;
            stored[4 * u + i] = here && t < sq.ctx;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const bool seen = stored[4 * u + i] && t <= pos[n] &&
                                (a.window == 0 || t > pos[n] - a.window || t < a.sinks);
              x[n][u][i] = seen ? x[n][u][i] : -INFINITY;
            }
          }
        }
      }
      // ---- scales of the values, pairs of keys; the running powers of two
      uint32_t sv[G][4], zv[G][4];
      f16x2_t most{0, 0};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x4 par[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          par[u] = *reinterpret_cast<const u32x4*>(slot + u * L::kBytes + 16 * D + G * 64 + g * 64 + 16 * kb);
        if (!whole || missing) {
#pragma unroll
          for (int e = 0; e < 8; ++e) par[e >> 2][e & 3] = stored[e] ? par[e >> 2][e & 3] : 0u;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t p0 = par[e >> 1][2 * (e & 1)], p1 = par[e >> 1][2 * (e & 1) + 1];
          zv[g][e] = (__builtin_amdgcn_perm(p1, p0, 0x0c060c02u) << 6) | magic_v;
          sv[g][e] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
          most = pk_max(most, __builtin_bit_cast(f16x2_t, sv[g][e]) * pair16(shrink[g]));
        }
      }
      bool grow = most[0] > static_cast<_Float16>(1.0f) || most[1] > static_cast<_Float16>(1.0f);
      if (__any(grow)) {       // some scale passed its 2^e
#pragma unroll
        for (int g = 0; g < G; ++g) {
          f16x2_t t{0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) t = pk_max(t, __builtin_bit_cast(f16x2_t, sv[g][e]));
          const float top = wave_max(fmaxf(static_cast<float>(t[0]), static_cast<float>(t[1])));
          // the largest scale to 2^-3 .. 2^-2; it only shrinks (a scale is below 2^16)
          const float next = fminf(shrink[g], __uint_as_float((251u - (__float_as_uint(top) >> 23)) << 23));
          const float f = next / shrink[g];
          shrink[g] = next;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            corr[n][g] *= f;
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= f;
          }
        }
      }
      // ---- running maximum
      grow = false;
      float top[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float t = fmaxf(fmaxf(x[n][0][0], x[n][0][1]), fmaxf(x[n][0][2], x[n][0][3]));
        t = fmaxf(t, fmaxf(fmaxf(x[n][1][0], x[n][1][1]), fmaxf(x[n][1][2], x[n][1][3])));
        top[n] = t;
        grow |= t > base[n] + 15.0f;
      }
      if (__any(grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          // 2^7 at the new maximum; rows that have seen no key stay at -inf
          const float next = fmaxf(base[n], max_over_quads(top[n]) - 7.0f);
          const float fade = next == -INFINITY ? 1.0f : exp2_fast(base[n] - next);
          base[n] = next;
          l[n] *= fade;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            corr[n][g] *= fade;
#pragma unroll
            for (int y = 0; y < MT; ++y) o[n][g][y] *= fade;
          }
        }
      }
      f16x2_t p[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float from = base[n] == -INFINITY ? 0.0f : base[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = exp2_fast(x[n][e >> 1][2 * (e & 1)] - from);
          const float p1 = exp2_fast(x[n][e >> 1][2 * (e & 1) + 1] - from);
          l[n] += p0 + p1;
          p[n][e] = f16x2_t{static_cast<_Float16>(p0), static_cast<_Float16>(p1)};
        }
      }
      // ---- values
#pragma unroll
      for (int g = 0; g < G; ++g) {
        u32x4 vw[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          vw[u] = *reinterpret_cast<const u32x4*>(slot + u * L::kBytes + 8 * D + kb * 2 * D +
                                                  16 * (g * (GROUP / 8) + (r & (GROUP / 8 - 1))));
        u32x4 pv[NT];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2_t s = __builtin_bit_cast(f16x2_t, sv[g][e]) * pair16(shrink[g]);
#pragma unroll
          for (int n = 0; n < NT; ++n) pv[n][e] = __builtin_bit_cast(uint32_t, p[n][e] * s);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) corr[n][g] = mfma_q<QMM_F16>(zv[g], pv[n], corr[n][g]);
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
            uint32_t av[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              av[e] = ((y < 2 ? unit[e] << (6 - 4 * y) : unit[e] >> (4 * y - 6)) & kNibbles) | magic_v;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              o[n][g][part * (MT / kParts) + y] = mfma_q<QMM_F16>(av, pv[n], o[n][g][part * (MT / kParts) + y]);
          }
        }
      }
    };

    // ---- steps, two requested ahead
    if (s_lo < s_hi) issue(st.key(s_lo), pages_of(st.key(s_lo)), 0);
    if (s_lo + kStride < s_hi) issue(st.key(s_lo + kStride), pages_of(st.key(s_lo + kStride)), 1);
    Pages pages = pages_of(st.key(s_lo + 2 * kStride));
    int stage = 0;
    for (int s = s_lo; s < s_hi; s += kStride) {
      const int ahead = stage == 0 ? 2 : stage - 1;
      __builtin_amdgcn_sched_barrier(0);
      if (s + 2 * kStride < s_hi) {
        issue(st.key(s + 2 * kStride), pages, ahead);
        pages = pages_of(st.key(s + 3 * kStride));
        wait_vm<2 * L::kLoads>();
      } else if (s + kStride < s_hi) {
        wait_vm<L::kLoads>();
      } else {
        wait_vm<0>();
      }
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      compute(st.key(s), stage);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);      // LDS reads of this stage done before it is requested again
      stage = stage == 2 ? 0 : stage + 1;
    }

    // ---- results: o - corr, joined over the wavefronts (WS), then out or the workspace
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] = sum_over_quads(l[n]);
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int y = 0; y < MT; ++y) o[n][g][y] = (o[n][g][y] - corr[n][g]) * (1.0f / shrink[g]);
    }
    // channel of row 4 kb + i of tile y of group g
    auto channel = [&](int g, int y, int i) {
      const int q = 4 * kb + i;
      if constexpr (GROUP == 128) return g * 128 + 8 * q + (y < 4 ? 2 * y : 2 * y - 7);
      else if constexpr (GROUP == 64) return g * 64 + 8 * (q & 7) + 2 * y + (q >> 3);
      else return g * 32 + 8 * (q & 3) + 4 * ((q >> 2) & 1) + 2 * y + (q >> 3);
    };
    float* lds = reinterpret_cast<float*>(&ring[0][0][0]);
    constexpr int kPad = D + 4;
    if constexpr (WS) {
      // one row tile at a time: maxima and sums of the four wavefronts, then their scaled sums
      static_assert(kWaves * 16 * kPad * 4 + kWaves * 32 * 4 <= kWaves * kStages * L::kStepBytes, "LDS");
      float* stat = lds + kWaves * 16 * kPad;
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
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, stat[w * 32 + r]);
        const float f = base[n] == -INFINITY ? 0.0f : exp2_fast(base[n] - mm);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) lds[(wave * 16 + r) * kPad + channel(g, y, i)] = o[n][g][y][i] * f;
        __syncthreads();
        constexpr int kPer = 16 * D / 256;     // channels per thread: kPer consecutive ones of a row
        const int rr = threadIdx.x / (256 / 16), c0 = (threadIdx.x % 16) * kPer;
        const int row = row_lo + 16 * n + rr;
        if (row < rows) {
          float M = -INFINITY, sum = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) M = fmaxf(M, stat[w * 32 + rr]);
#pragma unroll
          for (int w = 0; w < kWaves; ++w)
            sum += stat[w * 32 + rr] == -INFINITY ? 0.0f : stat[w * 32 + 16 + rr] * exp2_fast(stat[w * 32 + rr] - M);
          const int tok = row / a.ratio, head = kvh * a.ratio + row - tok * a.ratio;
          const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + head;
          const float inv = chunks > 1 ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
          float v[kPer];
#pragma unroll
          for (int c = 0; c < kPer; ++c) {
            v[c] = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v[c] += lds[(w * 16 + rr) * kPad + c0 + c];
            v[c] *= inv;
          }
          if (chunks > 1) {
            float* po = a.part_o + (rh * a.splits + split) * D + c0;
#pragma unroll
            for (int c = 0; c < kPer; c += 4) *reinterpret_cast<f32x4*>(po + c) = f32x4{v[c], v[c + 1], v[c + 2], v[c + 3]};
            if (c0 == 0) a.part_ml[rh * a.splits + split] = make_float2(M, sum);
          } else {
            uint16_t* po = a.out + rh * D + c0;
#pragma unroll
            for (int c = 0; c < kPer; c += 4)
              *reinterpret_cast<u32x2*>(po + c) = u32x2{pack2<DT>(v[c], v[c + 1]), pack2<DT>(v[c + 2], v[c + 3])};
            if (a.lse && c0 == 0) a.lse[rh] = sum > 0.0f ? (M + __builtin_amdgcn_logf(sum)) * 0.69314718055994531f : -INFINITY;
          }
        }
      }
    } else {
      // a wavefront's own rows: through its part of LDS, for whole 16-byte stores
      static_assert(16 * kPad * 4 <= kStages * L::kStepBytes, "LDS");
      float* mine = reinterpret_cast<float*>(&ring[wave][0][0]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        asm volatile("" ::: "memory");
        const float inv = l[n] > 0.0f ? 1.0f / l[n] : 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) mine[r * kPad + channel(g, y, i)] = o[n][g][y][i] * inv;
        asm volatile("" ::: "memory");
        const int row = row_lo + 16 * n + r;
        const int tok = row / a.ratio, head = kvh * a.ratio + row - tok * a.ratio;
        const int64_t rh = static_cast<int64_t>(sq.row0 + tok) * a.q_heads + head;
        if (row < rows && a.lse && kb == 0)
          a.lse[rh] = l[n] > 0.0f ? (base[n] + __builtin_amdgcn_logf(l[n])) * 0.69314718055994531f : -INFINITY;
        if (row < rows) {
#pragma unroll
          for (int c = 0; c < D / 4; c += 8) {
            const float* v = mine + r * kPad + kb * (D / 4) + c;
            *reinterpret_cast<u32x4*>(a.out + rh * D + kb * (D / 4) + c) =
                u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
          }
        }
        asm volatile("" ::: "memory");
      }
    }
    if (tile * kRows + a.row_tiles * kRows < rows) __syncthreads();   // LDS is free for the next rows
  }
}

template <int DT, int D, int GROUP, int NT, bool WS>
__global__ __launch_bounds__(256) void attention_kernel(AttnArgs a) {
  attention_block<DT, D, GROUP, NT, WS>(a);
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
    for (int c = lane; c < chunks; c += kWave) l += ml[c].x == -INFINITY ? 0.0f : ml[c].y * exp2_fast(ml[c].x - m);
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
      o *= l > 0.0f ? 1.0f / l : 0.0f;
      *reinterpret_cast<u32x2*>(a.out + rh * D + 4 * c4) = u32x2{pack2<DT>(o.x, o.y), pack2<DT>(o.z, o.w)};
      if (a.lse && c4 == 0) a.lse[rh] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

// ---- launch shape ------------------------------------------------------------
struct Plan {
  int nt;             // 16-row tiles a wavefront takes
  bool ws;            // wavefronts of a block share the rows and split the keys
  int64_t rows, row_tiles, splits, chunk;
};

Plan plan_of(int64_t seqs, int64_t max_q, int64_t ratio, int64_t kv_heads, int64_t D, int64_t max_context,
             int64_t window, int64_t sinks) {
  Plan p{};
  const int64_t rows = max_q * ratio;
  p.ws = rows <= 64;
  p.nt = rows <= 16 || D == 256 ? 1 : 2;
  p.rows = 16 * p.nt * (p.ws ? 1 : kWaves);
  p.row_tiles = std::min<int64_t>(ceil_div(rows, p.rows), 65535);
  int64_t steps = ceil_div(max_context, kStep);
  if (window > 0)
    steps = std::min(steps, ceil_div(std::min(window, max_context) + p.rows / ratio + 1, kStep) + 1 +
                                ceil_div(std::min(sinks, max_context), kStep));
  p.chunk = steps;
  if (p.ws) {
    const int64_t blocks = seqs * kv_heads * p.row_tiles;
    const int64_t want = std::max<int64_t>(1, 2048 / blocks);
    p.chunk = std::max<int64_t>(ceil_div(steps, want), 8);
  }
  p.splits = std::max<int64_t>(1, ceil_div(steps, p.chunk));
  return p;
}

size_t workspace_bytes_of(const Plan& p, int64_t T, int64_t q_heads, int64_t D) {
  return p.splits > 1 ? static_cast<size_t>(T) * q_heads * p.splits * (D + 2) * 4 : 0;
}

template <int DT, int D, int GROUP>
void launch(const AttnArgs& a, const Plan& p, unsigned blocks, hipStream_t s) {
  constexpr int kMost = D == 256 ? 1 : 2;
  if (!p.ws) attention_kernel<DT, D, GROUP, kMost, false><<<blocks, 256, 0, s>>>(a);
  else if (p.nt == 1) attention_kernel<DT, D, GROUP, 1, true><<<blocks, 256, 0, s>>>(a);
  else attention_kernel<DT, D, GROUP, kMost, true><<<blocks, 256, 0, s>>>(a);
}

template <int DT>
void launch_dt(const AttnArgs& a, const Plan& p, unsigned blocks, hipStream_t s) {
  const int D = a.sh.D, g = a.sh.group;
  if (D == 64) {
    if (g == 32) launch<DT, 64, 32>(a, p, blocks, s); else launch<DT, 64, 64>(a, p, blocks, s);
  } else if (D == 128) {
    if (g == 32) launch<DT, 128, 32>(a, p, blocks, s);
    else if (g == 64) launch<DT, 128, 64>(a, p, blocks, s);
    else launch<DT, 128, 128>(a, p, blocks, s);
  } else {
    if (g == 32) launch<DT, 256, 32>(a, p, blocks, s);
    else if (g == 64) launch<DT, 256, 64>(a, p, blocks, s);
    else launch<DT, 256, 128>(a, p, blocks, s);
  }
  if (p.splits > 1) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(p.row_tiles * p.rows, a.ratio), 1024)),
                    static_cast<unsigned>(a.q_heads), static_cast<unsigned>(a.seqs));
    const int rows = static_cast<int>(p.rows);
    if (D == 64) attention_join_kernel<DT, 64><<<grid, 256, 0, s>>>(a, rows);
    else if (D == 128) attention_join_kernel<DT, 128><<<grid, 256, 0, s>>>(a, rows);
    else attention_join_kernel<DT, 256><<<grid, 256, 0, s>>>(a, rows);
  }
}

}  // namespace
}  // namespace qmm

extern "C" size_t kv4_attention_workspace_bytes(int64_t T, int64_t seqs, int64_t max_q, int64_t q_heads,
                                                int64_t kv_heads, int64_t head_dim, int64_t max_context,
                                                int64_t window, int64_t sinks) {
  using namespace qmm;
  if (T <= 0 || seqs <= 0 || max_q <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0 ||
      max_context <= 0 || max_context >= (int64_t{1} << 31) || window < 0 || sinks < 0 || T >= (int64_t{1} << 31) ||
      seqs > 65535 || q_heads > 65535)
    return 0;
  return workspace_bytes_of(plan_of(seqs, std::min(max_q, T), q_heads / kv_heads, kv_heads, head_dim, max_context,
                                    window, sinks), T, q_heads, head_dim);
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
  const Plan p = plan_of(seqs, cu_q ? std::min(max_q, T) : 1, ratio, kv_heads, head_dim, tokens, window, sinks);
  const size_t need = workspace_bytes_of(p, T, q_heads, head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return QMM_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 16)) return QMM_EALIGN;
  const int64_t blocks = seqs * kv_heads * p.row_tiles * p.splits;
  if (blocks >= (int64_t{1} << 31)) return QMM_ERANGE;
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
  if (dtype == QMM_BF16) launch_dt<QMM_BF16>(a, p, static_cast<unsigned>(blocks), as_stream(stream));
  else launch_dt<QMM_F16>(a, p, static_cast<unsigned>(blocks), as_stream(stream));
  return launch_status();
}
