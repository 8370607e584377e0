// beams.hip -- beam search over the 4-bit cache: which beams go on with which
// tokens, and the reordering of their pages (definitions: include/qmm.h).

#include <algorithm>

#include "kv4_device.h"

namespace qmm {
namespace {

typedef short i16x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_anywhere __attribute__((aligned(2)));

constexpr int kMostBeams = 64, kMostK = 64;
constexpr int kThreadBytes = 128;                  // logits of a thread

// What a block found in its logits of a row: their maximum and the sum of
// exp(x - maximum).
struct Partial {
  double sum;
  float most;
  float unused;
};
struct Candidate {
  float x;
  uint32_t token;
};

// Numbers in their order as unsigned ones (-0 first made 0).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The k-th and the few-th largest key of the wavefront's lanes (0: not so many
// are not 0), few <= k.  Two searches at once: each waits for its own counts.
__device__ __forceinline__ void kth_largest(uint32_t key, int bits, int k, int few, uint32_t* at_k, uint32_t* at_few) {
  uint32_t a = 0, b = 0;
  for (int bit = bits - 1; bit >= 0; --bit) {
    const uint32_t next_a = a | 1u << bit, next_b = b | 1u << bit;
    if (__popcll(__ballot(key >= next_a)) >= k) a = next_a;
    if (__popcll(__ballot(key >= next_b)) >= few) b = next_b;
  }
  *at_k = a;
  *at_few = b;
}

// A key below which no value is among the k best (0: no bound): the k-th best of
// the lanes' best ones.  But for equal keys at most k lanes of a wavefront hold
// values that it lets through.  A wavefront's by its k best lanes and by its share
// of k best of the block's; what the block then goes by: the tightest of the first
// or the loosest of the second, which lets through k lanes of all together and is
// the tighter one but for few or sorted values.
struct Bounds {
  uint32_t k, share;
};
__device__ __forceinline__ Bounds bounds_of(uint32_t best, int bits, int k, int waves) {
  Bounds b;
  kth_largest(best, bits, k, (k + waves - 1) / waves, &b.k, &b.share);
  return b;
}
template <int WAVES>
__device__ __forceinline__ uint32_t block_bound(const Bounds (&all)[WAVES]) {
  uint32_t most = all[0].k, least = all[0].share;
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    most = max(most, all[w].k);
    least = min(least, all[w].share);
  }
  return max(most, least);
}
// Candidates that a wavefront has room for.
__host__ __device__ constexpr int room_of(int k) { return 2 * k + 32; }

__device__ __forceinline__ double wave_sum(double v) {
  v += dpp_d<kDppXor1>(v);
  v += dpp_d<kDppXor2>(v);
  v += dpp_d<kDppHalfMirror>(v);
  v += dpp_d<kDppMirror>(v);
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

struct Select {
  const void* logits;
  int64_t row_stride;
  int64_t rows;
  int32_t vocabulary, beams, k, chunks;
  const float* scores;
  const uint8_t* finished;   // may be null
  int32_t pad;
  Partial* partial;          // [rows][chunks]
  Candidate* list;           // [rows][chunks][k]
  float* out_scores;
  int64_t* out_tokens;
  int64_t* out_parents;
};

// The largest of 16-bit floating-point numbers by their bits: as whole numbers
// with a sign the positive ones stand in their order, the negative ones in the
// opposite one.
template <int N>
__device__ __forceinline__ uint32_t largest_bits(const u32x4 (&v)[N]) {
  i16x2 most = __builtin_bit_cast(i16x2, static_cast<uint32_t>(v[0][0])), least = most;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t u = v[j][w];
      most = __builtin_elementwise_max(most, __builtin_bit_cast(i16x2, u));
      least = __builtin_elementwise_min(least, __builtin_bit_cast(i16x2, u));
    }
  const int m = max(most[0], most[1]), l = min(least[0], least[1]);
  return static_cast<uint32_t>(m >= 0 ? m : l) & 0xFFFFu;
}

template <int DT>
struct Logits;               // 16-byte pieces of a row
template <>
struct Logits<QMM_F32> {
  static constexpr int kOf = 4, kBits = 32;                  // numbers of a piece, bits of one
  static constexpr uint32_t kNone = 0xFF800000u;             // -inf
  // the type's numbers in their order as unsigned ones (never 0 above -inf)
  static __device__ __forceinline__ uint32_t key(float x) { return ordered(x); }
  template <int N>
  static __device__ __forceinline__ float largest(const u32x4 (&v)[N]) {
    float most = -INFINITY;                                  // (a NaN makes it wrong, and is found in the sum)
#pragma unroll
    for (int j = 0; j < N; ++j) most = max3(max3(most, get(v[j], 0), get(v[j], 1)), get(v[j], 2), get(v[j], 3));
    return most;
  }
  static __device__ __forceinline__ float value(uint32_t k) { return unordered(k); }
  static __device__ __forceinline__ float get(u32x4 v, int e) { return __uint_as_float(v[e]); }
  static __device__ __forceinline__ void set_none(u32x4& v, int e) { v[e] = kNone; }
};
template <>
struct Logits<QMM_BF16> {
  static constexpr int kOf = 8, kBits = 16;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  static __device__ __forceinline__ uint32_t key(float x) { return ordered(x) >> 16; }
  template <int N>
  static __device__ __forceinline__ float largest(const u32x4 (&v)[N]) { return bf16lo_to_f32(largest_bits(v)); }
  static __device__ __forceinline__ float value(uint32_t k) { return bf16hi_to_f32(__float_as_uint(unordered(k << 16 | (k & 0x8000u ? 0u : 0xFFFFu)))); }
  static __device__ __forceinline__ float get(u32x4 v, int e) {
    return e & 1 ? bf16hi_to_f32(v[e / 2]) : bf16lo_to_f32(v[e / 2]);
  }
  static __device__ __forceinline__ void set_none(u32x4& v, int e) {
    v[e / 2] = e & 1 ? (v[e / 2] & 0xFFFFu) | 0xFF800000u : (v[e / 2] & 0xFFFF0000u) | 0xFF80u;
  }
};
template <>
struct Logits<QMM_F16> {
  static constexpr int kOf = 8, kBits = 16;
  static constexpr uint32_t kNone = 0xFC00FC00u;
  template <int N>
  static __device__ __forceinline__ float largest(const u32x4 (&v)[N]) { return f16lo_to_f32(largest_bits(v)); }
  static __device__ __forceinline__ uint32_t key(float x) {
    const uint32_t u = f32_to_f16_bits(x + 0.0f);
    return u & 0x8000u ? ~u & 0xFFFFu : u | 0x8000u;
  }
  static __device__ __forceinline__ float value(uint32_t k) { return f16lo_to_f32(k & 0x8000u ? k ^ 0x8000u : ~k); }
  static __device__ __forceinline__ float get(u32x4 v, int e) {
    return e & 1 ? f16hi_to_f32(v[e / 2]) : f16lo_to_f32(v[e / 2]);
  }
  static __device__ __forceinline__ void set_none(u32x4& v, int e) {
    v[e / 2] = e & 1 ? (v[e / 2] & 0xFFFFu) | 0xFC000000u : (v[e / 2] & 0xFFFF0000u) | 0xFC00u;
  }
};

// A block takes 8192 fp32 logits of a row or 16384 of 16 bits, 128 bytes a thread
// in registers, reads them once and finds their maximum, the sum of exponentials
// and the k largest.  The largest: no logit below the k-th best of a wavefront's
// 64 lane maxima can be among them (a search over the bits of a key, one
// comparison and a count of lanes each), so a few more than k reach LDS, where
// each counts those before it.  These, which are most of a peaked row's sum, add
// to it in fp64, the others in fp32 by the hardware's exponential: two beams'
// candidates that are nearly as good are told apart by their rows' sums.
//   Where values equal to the bound, or sorted ones, are more than LDS has room
// for, or a NaN is met (the sum has taken it), the k largest are found one by one.
//   64 x 8 rows of 131072 bf16 logits 42 us, 3.2 TB/s: bound by vector operations,
// about ten a logit (unpacking, maximum, exponential at a quarter of the rate, sum,
// comparison).  With 64 bytes of logits a thread the call took 67 us instead of
// 60.6: its searches come twice as often.
template <int DT>
__global__ __launch_bounds__(256, 5) void beam_rows_kernel(Select a) {
  using L = Logits<DT>;
  constexpr int kOf = L::kOf, kPieces = kThreadBytes / 16;
  constexpr int kChunk = 256 * kPieces * kOf;
  constexpr float kLog2e = 1.44269504088896341f;
  extern __shared__ __attribute__((aligned(16))) float pool_x[];       // [4][room_of(k)], then as many tokens
  __shared__ float s_most[4], s_sum[4];
  __shared__ double s_large[4];
  __shared__ Bounds s_bound[4];
  __shared__ uint64_t s_best[4];
  __shared__ int s_rank[4][kWave];
  __shared__ int s_count[4], s_again[4];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int chunk = blockIdx.x;
  const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * 65535;
  if (row >= a.rows || (a.finished && a.finished[row])) return;
  const int room = room_of(a.k);
  uint32_t* const pool_token = reinterpret_cast<uint32_t*>(pool_x + 4 * room);

  // Whole pieces from the row's start on, wherever that lies (the hardware takes
  // 16 bytes from any address, and rows of the same logits have the same sums to
  // the last bit), and what is left behind them for the first threads.
  constexpr int kSize = 16 / kOf;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * kSize;
  const int pieces = a.vocabulary / kOf, behind = a.vocabulary % kOf;
  u32x4 raw[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int p = (chunk * kPieces + j) * 256 + tid;
    raw[j] = u32x4{L::kNone, L::kNone, L::kNone, L::kNone};
    if (p < pieces) raw[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_anywhere*>(base + static_cast<int64_t>(p) * 16));
  }
  uint32_t first_index = static_cast<uint32_t>(chunk * kChunk + tid * kOf);
  auto index_of = [&](int j, int e) { return first_index + static_cast<uint32_t>(j * 256 * kOf + e); };
  float odd = -INFINITY;
  uint32_t odd_index = 0;
  if (chunk == 0 && tid < behind) {
    odd_index = a.vocabulary - behind + tid;
    if constexpr (DT == QMM_F32) odd = reinterpret_cast<const float*>(base)[odd_index];
    else if constexpr (DT == QMM_BF16) odd = bf16lo_to_f32(reinterpret_cast<const uint16_t*>(base)[odd_index]);
    else odd = f16lo_to_f32(reinterpret_cast<const uint16_t*>(base)[odd_index]);
  }

  // ---- the lane's best, the block's maximum, the bound
  const float best = fmaxf(L::largest(raw), odd);
  const Bounds mine = bounds_of(best > -INFINITY ? L::key(best) : 0u, L::kBits, a.k, 4);
  float most = wave_max(best);
  if (lane == 0) {
    s_most[wave] = most;
    s_bound[wave] = mine;
  }
  __syncthreads();
  const uint32_t bound = block_bound(s_bound);
  most = fmaxf(fmaxf(s_most[0], s_most[1]), fmaxf(s_most[2], s_most[3]));
  // ---- sums below the bound; what passes it (without one all but -inf does)
  // goes to the wavefront's part of LDS
  const float least = bound ? L::value(bound) : -3.402823466e38f;
  const float at_base = most == -INFINITY ? 0.0f : most * kLog2e;
  float sum = 0.0f;
  int mine_n = 0;
  auto term = [&](float x) { return __builtin_amdgcn_exp2f(fmaf(x, kLog2e, -at_base)); };
  constexpr int kNotGreaterOrEqual = 12;                   // (the compiler's number of that comparison, true for NaN)
  auto take = [&](float x, uint32_t at, uint64_t who) {
    const int n = mine_n + static_cast<int>(__builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(who >> 32),
                                                                      __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(who), 0u)));
    if (x >= least && n < room) {
      pool_x[wave * room + n] = x;
      pool_token[wave * room + n] = at;
    }
    mine_n += __popcll(who);
  };
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    asm volatile("" : "+v"(raw[j]), "+v"(first_index));    // numbers are unpacked where they are used, indexes worked out
    uint64_t below[kOf], all = ~uint64_t{0};               // lanes, NaN among them
    float x[kOf];
#pragma unroll
    for (int e = 0; e < kOf; ++e) {
      x[e] = L::get(raw[j], e);
      below[e] = __builtin_amdgcn_fcmpf(x[e], least, kNotGreaterOrEqual);
      all &= below[e];
      sum += __builtin_amdgcn_inverse_ballot_w64(below[e]) ? term(x[e]) : 0.0f;
    }
    if (~all) {
#pragma unroll
      for (int e = 0; e < kOf; ++e)
        if (~below[e]) take(x[e], index_of(j, e), ~below[e]);
    }
  }
  sum += odd >= least ? 0.0f : term(odd);
  if (const uint64_t who = __ballot(odd >= least)) take(odd, odd_index, who);
  const bool nan = __any(sum != sum);
  sum = wave_sum(sum);
  if (lane == 0) {
    // (past 2^24 the rounding of at_base is no small number)
    s_again[wave] = nan || mine_n > room || fabsf(most) > 0x1p24f;
    s_count[wave] = mine_n;
    s_sum[wave] = sum;
  }
  __syncthreads();

  const int64_t at = row * a.chunks + chunk;
  Candidate* list = a.list + at * a.k;
  double small, large = 0.0;          // the sums of those that were not and those that were taken
  double back;                        // from the first's base to the maximum
  if (!(s_again[0] | s_again[1] | s_again[2] | s_again[3])) {
    // each candidate counts those before it
    const int n1 = s_count[0], n2 = n1 + s_count[1], n3 = n2 + s_count[2], n = n3 + s_count[3];
    auto place_of = [&](int i) { return i < n1 ? i : i < n2 ? room + i - n1 : i < n3 ? 2 * room + i - n2 : 3 * room + i - n3; };
    // (of few, every wavefront counts among its own)
    if (n <= kWave) {
      if (lane < n) {
        const float x = pool_x[place_of(lane)];
        const uint32_t key = ordered(x), token = pool_token[place_of(lane)];
        int rank = 0;
        const int count = s_count[wave];
#pragma unroll 4
        for (int j = 0; j < count; ++j) {
          const uint32_t ko = ordered(pool_x[wave * room + j]);
          rank += ko > key || (ko == key && pool_token[wave * room + j] < token);
        }
        s_rank[wave][lane] = rank;
      }
      __syncthreads();
      if (tid < n) {
        const int rank = s_rank[0][tid] + s_rank[1][tid] + s_rank[2][tid] + s_rank[3][tid];
        const Candidate c{pool_x[place_of(tid)], pool_token[place_of(tid)]};
        if (rank < a.k) list[rank] = c;
        large = exp(static_cast<double>(c.x) - static_cast<double>(most));
      }
    } else for (int i = tid; i < n; i += 256) {
      const int place = place_of(i);
      const Candidate c{pool_x[place], pool_token[place]};
      const uint32_t key = ordered(c.x);
      int rank = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int count = s_count[w];
#pragma unroll 4
        for (int j = 0; j < count; ++j) {
          const uint32_t ko = ordered(pool_x[w * room + j]);
          rank += ko > key || (ko == key && pool_token[w * room + j] < c.token);
        }
      }
      if (rank < a.k) list[rank] = c;
      large += exp(static_cast<double>(c.x) - static_cast<double>(most));
    }
    for (int i = n + tid; i < a.k; i += 256) list[i] = {-INFINITY, 0u};
    if (wave == 0 || n > kWave) large = wave_sum(large);     // (64 or fewer are all the first's)
    small = static_cast<double>(s_sum[0]) + s_sum[1] + s_sum[2] + s_sum[3];
    back = 0.0;
  } else {
    // ---- one by one, in their order: the largest below the last one taken, of
    // logits read again (registers would hold them for this path alone)
    auto each = [&](auto&& f) {
      f(odd, odd_index);
#pragma unroll 1
      for (int j = 0; j < kPieces; ++j) {
        const int p = (chunk * kPieces + j) * 256 + tid;
        if (p >= pieces) break;
        const u32x4 v = *reinterpret_cast<const u32x4_anywhere*>(base + static_cast<int64_t>(p) * 16);
#pragma unroll
        for (int e = 0; e < kOf; ++e) f(L::get(v, e), static_cast<uint32_t>(p * kOf + e));
      }
    };
    auto key_of = [](float x, uint32_t index) { return static_cast<uint64_t>(ordered(x)) << 32 | static_cast<uint32_t>(~index); };
    auto best_below = [&](uint64_t last) {
      uint64_t top = 0;               // key, then the index the other way round; 0: none
      each([&](float x, uint32_t index) {
        const uint64_t key = key_of(x, index);
        if (x > -INFINITY && key < last) top = max(top, key);
      });
#pragma unroll 1
      for (int i = 1; i < kWave; i <<= 1)
        top = max(top, static_cast<uint64_t>(__shfl_xor(static_cast<long long>(top), i, kWave)));
      __syncthreads();
      if (lane == 0) s_best[wave] = top;
      __syncthreads();
      return max(max(s_best[0], s_best[1]), max(s_best[2], s_best[3]));
    };
    uint64_t last = ~uint64_t{0};
    most = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < a.k; ++i) {
      const uint64_t next = last ? best_below(last) : 0;
      const float x = next ? unordered(static_cast<uint32_t>(next >> 32)) : -INFINITY;
      if (i == 0) most = x;
      if (tid == 0) list[i] = {x, next ? ~static_cast<uint32_t>(next) : 0u};
      if (next && tid == 0) large += exp(static_cast<double>(x) - static_cast<double>(most));
      last = next;
    }
    const float from = most == -INFINITY ? 0.0f : most;
    sum = 0.0f;
    each([&](float x, uint32_t index) {
      if (x > -INFINITY && key_of(x, index) < last) sum += __builtin_amdgcn_exp2f((x - from) * kLog2e);
    });
    sum = wave_sum(sum);
    __syncthreads();
    if (lane == 0) s_sum[wave] = sum;
    __syncthreads();
    small = static_cast<double>(s_sum[0]) + s_sum[1] + s_sum[2] + s_sum[3];
    back = 1.0;
  }
  if (lane == 0) s_large[wave] = large;
  __syncthreads();
  if (tid == 0) {
    // the fp32 terms' own base back to the maximum: what its rounding left
    if (back == 0.0) back = exp2(static_cast<double>(at_base) - static_cast<double>(most) * static_cast<double>(kLog2e));
    if (most == -INFINITY) back = 1.0;
    a.partial[at] = {fma(small, back, s_large[0] + s_large[1] + s_large[2] + s_large[3]), most, 0.0f};
  }
}

// A block joins the rows of a sequence: each beam's log sum, then the k best of
// the blocks' candidates, 2048 at a time, by the same bound.  Values are fp64, the
// bound is by fp32 keys: all that round to the bound's pass.  There is room for
// every candidate that is looked at; they come to it in any order, and each counts
// those before it by value and index.
//   One block to a sequence: 64 x 8 rows 12 us, a chain of loads, searches and
// barriers.
constexpr int kJoinThreads = 512, kJoinWaves = kJoinThreads / kWave, kJoinPer = 4;
constexpr int kJoinRoom = kJoinThreads * kJoinPer + kMostK;            // and the ones kept

__global__ __launch_bounds__(kJoinThreads) void beam_join_kernel(Select a) {
  __shared__ double s_offset[kMostBeams];
  __shared__ int s_alive[kMostBeams];
  __shared__ Bounds s_bound[kJoinWaves];
  __shared__ int s_count;
  __shared__ double value[kJoinRoom], kept_value[kMostK];
  __shared__ uint32_t place[kJoinRoom], kept_place[kMostK];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.beams;
  const int total = a.beams * a.chunks * a.k, row_of = a.chunks * a.k;
  // the first candidates are on their way while the sums are joined
  Candidate c[kJoinPer];
  auto fetch = [&](int first) {
#pragma unroll
    for (int i = 0; i < kJoinPer; ++i) {
      const int e = first + i * kJoinThreads + tid;
      c[i] = e < total ? a.list[row0 * row_of + e] : Candidate{-INFINITY, 0u};
    }
  };
  fetch(0);
  for (int b = wave; b < a.beams; b += kJoinWaves) {
    const float score = a.scores[row0 + b];
    const bool ends = a.finished && a.finished[row0 + b];
    double offset = 0.0;
    bool alive = fabsf(score) < INFINITY;
    if (!ends) {
      const Partial* p = a.partial + (row0 + b) * a.chunks;
      float most = -INFINITY;
      double sum = 0.0;
      for (int i = 0; i < a.chunks; i += kWave) {            // (64 blocks hold most vocabularies)
        const Partial mine = i + lane < a.chunks ? p[i + lane] : Partial{0.0, -INFINITY, 0.0f};
        const float now = fmaxf(most, wave_max(mine.most));
        if (now > most) sum *= exp(static_cast<double>(most) - static_cast<double>(now));
        most = now;
        if (mine.most > -INFINITY) sum += mine.sum * exp(static_cast<double>(mine.most) - static_cast<double>(most));
      }
      sum = wave_sum(sum);
      offset = static_cast<double>(score) - (static_cast<double>(most) + log(sum));
      alive = alive && fabsf(most) < INFINITY;
    }
    if (lane == 0) {
      s_offset[b] = offset;
      s_alive[b] = alive ? (ends ? 2 : 1) : 0;
    }
  }
  __syncthreads();

  const double per_row = 1.0 / row_of;
  int kept = 0;
  for (int first = 0; first < total; first += kJoinThreads * kJoinPer) {
    if (first > 0) fetch(first);
    double v[kJoinPer];
    uint32_t at[kJoinPer];
    double best = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < kJoinPer; ++i) {
      const int e = first + i * kJoinThreads + tid;
      v[i] = -__builtin_inf();
      at[i] = 0;
      if (e < total) {
        const int b = static_cast<int>((e + 0.5) * per_row), alive = s_alive[b];      // e / row_of
        at[i] = static_cast<uint32_t>(b) * a.vocabulary;
        if (alive == 1) {
          v[i] = s_offset[b] + static_cast<double>(c[i].x);
          at[i] += c[i].token;
        } else if (alive == 2 && e == b * row_of) {            // a finished beam's one
          v[i] = a.scores[row0 + b];
          at[i] += a.pad;
        }
      }
      best = fmax(best, v[i]);
    }
    const Bounds mine = bounds_of(best > -__builtin_inf() ? ordered(static_cast<float>(best)) : 0u, 32, a.k, kJoinWaves);
    if (lane == 0) s_bound[wave] = mine;
    for (int i = tid; i < kept; i += kJoinThreads) {           // the best of those before
      value[i] = kept_value[i];
      place[i] = kept_place[i];
    }
    if (tid == 0) s_count = kept;
    __syncthreads();
    const uint32_t bound = block_bound(s_bound);
#pragma unroll
    for (int i = 0; i < kJoinPer; ++i) {
      if (v[i] > -__builtin_inf() && ordered(static_cast<float>(v[i])) >= bound) {
        const int n = atomicAdd(&s_count, 1);
        value[n] = v[i];
        place[n] = at[i];
      }
    }
    __syncthreads();
    const int n = s_count;
    kept = min(n, a.k);
    for (int i = tid; i < n; i += kJoinThreads) {
      const double mine_v = value[i];
      const uint32_t mine_at = place[i];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) rank += value[j] > mine_v || (value[j] == mine_v && place[j] < mine_at);
      if (rank < a.k) {
        kept_value[rank] = mine_v;
        kept_place[rank] = mine_at;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < a.k; i += kJoinThreads) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * a.k + i;
    const bool some = i < kept;
    const uint32_t at = some ? kept_place[i] : 0u, b = at / a.vocabulary;
    a.out_scores[o] = some ? static_cast<float>(kept_value[i]) : -INFINITY;
    a.out_tokens[o] = some ? static_cast<int64_t>(at - b * a.vocabulary) : -1;
    a.out_parents[o] = some ? b : i % a.beams;
  }
}

int64_t chunks_of(int64_t vocabulary, int bytes) { return ceil_div(vocabulary, 256 * kThreadBytes / bytes); }

size_t select_bytes(int64_t rows, int64_t vocabulary, int64_t k) {
  return static_cast<size_t>(rows) * chunks_of(vocabulary, 4) * (sizeof(Partial) + k * sizeof(Candidate));
}

// ---------------------------------------------------------------------------
// Reordering of the beams' pages.
// ---------------------------------------------------------------------------
struct Reorder {
  uint8_t* cache;
  Kv4Shape sh;
  const int32_t* table;
  int32_t width;
  const int32_t* context;
  const int32_t* tails;      // [slots][2]
  const int64_t* parents;    // [slots], a beam of the slot's sequence
  int32_t beams;
  int32_t* table_out;
  int32_t* context_out;
};

// blockIdx.x a slot, .y a layer, .z two of its heads: the filled part of the
// parent's last page, four 16-byte pieces a thread in flight.  The first block
// of a slot writes its row of the table.  Bound by memory and, before the first
// piece, by four loads that wait for each other (parent, its length, its page,
// the piece): 16 x 8 beams in 16 layers of 8 heads of 128, 77 MB read and written,
// 33 us with all heads in a block, 28 with one, 24.5 with two.
constexpr int kReorderPieces = 4, kReorderHeads = 2;

__global__ __launch_bounds__(256) void kv4_beam_reorder_kernel(Reorder a) {
  const int slot = blockIdx.x, seq = slot / a.beams;
  const int64_t beam = a.parents[slot];
  const int parent = beam >= 0 && beam < a.beams ? seq * a.beams + static_cast<int>(beam) : slot;
  const int64_t most = static_cast<int64_t>(a.width) << a.sh.shift;
  const int n = static_cast<int>(min(max<int64_t>(a.context[parent], 0), most));
  const int own = static_cast<int>(min(max<int64_t>(a.context[slot], 0), most));
  const int32_t* theirs = a.table + static_cast<int64_t>(parent) * a.width;
  const int column = n >> a.sh.shift, filled = n & (a.sh.page - 1);
  const bool moved = parent != slot && filled != 0;
  int from = -1, to = -1;
  if (moved) {
    from = theirs[column];
    const int at = own >> a.sh.shift;
    const int mine = at < a.width ? a.table[static_cast<int64_t>(slot) * a.width + at] : -1;
    const int32_t t0 = a.tails[2 * slot], t1 = a.tails[2 * slot + 1];
    to = mine == t0 ? t1 : t0;
  }
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    int32_t* out = a.table_out + static_cast<int64_t>(slot) * a.width;
    for (int j = threadIdx.x; j < a.width; j += 256) out[j] = moved && j == column ? to : theirs[j];
    if (threadIdx.x == 0) a.context_out[slot] = n;
  }
  const uint32_t pages = static_cast<uint32_t>(a.sh.pages);
  if (!moved || static_cast<uint32_t>(from) >= pages || static_cast<uint32_t>(to) >= pages || from == to) return;

  // fours of tokens: pieces of K codes, of V codes, then of each row of params
  const int fours = (filled + 3) >> 2, D = a.sh.D;
  const int codes = fours * (D / 8), record = 2 * codes + 2 * a.sh.groups() * fours;
  const int h0 = static_cast<int>(blockIdx.z) * kReorderHeads, h1 = min(h0 + kReorderHeads, a.sh.heads);
  const float per_four = 1.0f / fours;
  const int64_t bytes = a.sh.record_bytes();
  uint8_t* layer = a.cache + static_cast<int64_t>(blockIdx.y) * a.sh.pages * a.sh.heads * bytes;
  const uint8_t* src = layer + static_cast<int64_t>(from) * a.sh.heads * bytes;
  uint8_t* dst = layer + static_cast<int64_t>(to) * a.sh.heads * bytes;
  const int total = (h1 - h0) * record;
  for (int p0 = threadIdx.x; p0 < total; p0 += kReorderPieces * 256) {
    u32x4 x[kReorderPieces];
    int64_t at[kReorderPieces];
#pragma unroll
    for (int i = 0; i < kReorderPieces; ++i) {
      const int p = p0 + i * 256;
      if (p < total) {
        const int h = p >= record ? 1 : 0, q = p - h * record;
        int offset = 16 * q;
        if (q >= 2 * codes) {
          const int r = static_cast<int>((q - 2 * codes + 0.5f) * per_four);          // (q - 2 codes) / fours
          offset = a.sh.page * (D + 4 * r) + 16 * (q - 2 * codes - r * fours);
        } else if (q >= codes) {
          offset = a.sh.page * (D / 2) + 16 * (q - codes);
        }
        at[i] = (h0 + h) * bytes + offset;
        x[i] = ld16_nt(src + at[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kReorderPieces; ++i)
      if (p0 + i * 256 < total) st16_nt(dst + at[i], x[i]);
  }
}

}  // namespace
}  // namespace qmm

extern "C" size_t beam_select_workspace_bytes(int64_t seqs, int64_t beams, int64_t vocabulary, int64_t k) {
  using namespace qmm;
  if (seqs <= 0 || beams <= 0 || vocabulary <= 0 || k <= 0 || beams > kMostBeams || k > kMostK ||
      vocabulary >= (int64_t{1} << 31) / beams || seqs >= (int64_t{1} << 24) / beams)
    return 0;
  return select_bytes(seqs * beams, vocabulary, k);
}

extern "C" int beam_select(const void* logits, int dtype, int64_t row_stride, int64_t seqs, int64_t beams,
                           int64_t vocabulary, const float* scores, const uint8_t* finished, int64_t pad, int64_t k,
                           float* out_scores, int64_t* out_tokens, int64_t* out_parents, void* workspace,
                           size_t workspace_bytes, void* stream) {
  using namespace qmm;
  if (seqs == 0) return QMM_OK;
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents || seqs < 0 || beams <= 0 || vocabulary <= 0 ||
      k <= 0 || row_stride < vocabulary || pad < 0 || pad >= vocabulary || dtype < QMM_F32 || dtype > QMM_I32)
    return QMM_EINVAL;
  if (dtype == QMM_I32 || beams > kMostBeams || k > kMostK) return QMM_EUNSUPPORTED;
  if (vocabulary >= (int64_t{1} << 31) / beams || seqs >= (int64_t{1} << 24) / beams) return QMM_ERANGE;
  const int64_t rows = seqs * beams, chunks = chunks_of(vocabulary, dtype == QMM_F32 ? 4 : 2);
  if (rows * chunks >= (int64_t{1} << 24)) return QMM_ERANGE;            // blocks of 256 threads a launch holds
  if (!aligned(logits, dtype == QMM_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
      !aligned(out_tokens, 8) || !aligned(out_parents, 8))
    return QMM_EALIGN;
  if (!workspace || workspace_bytes < select_bytes(rows, vocabulary, k)) return QMM_EWORKSPACE;
  if (!aligned(workspace, 16)) return QMM_EALIGN;
  Select a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.rows = rows;
  a.vocabulary = static_cast<int32_t>(vocabulary);
  a.beams = static_cast<int32_t>(beams);
  a.k = static_cast<int32_t>(k);
  a.chunks = static_cast<int32_t>(chunks);
  a.scores = scores;
  a.finished = finished;
  a.pad = static_cast<int32_t>(pad);
  a.partial = static_cast<Partial*>(workspace);
  a.list = reinterpret_cast<Candidate*>(a.partial + rows * chunks);
  a.out_scores = out_scores;
  a.out_tokens = out_tokens;
  a.out_parents = out_parents;
  hipStream_t s = as_stream(stream);
  const size_t lds = 4 * room_of(static_cast<int>(k)) * sizeof(Candidate);
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(std::min<int64_t>(rows, 65535)),
                  static_cast<unsigned>(ceil_div(rows, 65535)));
  if (dtype == QMM_BF16) beam_rows_kernel<QMM_BF16><<<grid, 256, lds, s>>>(a);
  else if (dtype == QMM_F16) beam_rows_kernel<QMM_F16><<<grid, 256, lds, s>>>(a);
  else beam_rows_kernel<QMM_F32><<<grid, 256, lds, s>>>(a);
  beam_join_kernel<<<static_cast<unsigned>(seqs), kJoinThreads, 0, s>>>(a);
  return launch_status();
}

extern "C" int kv4_beam_reorder(uint8_t* cache, int64_t layers, int64_t pages, int64_t kv_heads, int64_t head_dim,
                                int64_t page, int group, const int32_t* page_table, int64_t table_width,
                                const int32_t* context, const int32_t* tails, const int64_t* parents, int64_t seqs,
                                int64_t beams, int32_t* table_out, int32_t* context_out, void* stream) {
  using namespace qmm;
  if (seqs == 0) return QMM_OK;
  if (!cache || !page_table || !context || !tails || !parents || !table_out || !context_out || layers <= 0 ||
      table_width <= 0 || seqs < 0 || beams <= 0)
    return QMM_EINVAL;
  if (page_table == table_out || context == context_out) return QMM_EINVAL;
  Kv4Shape sh;
  if (const int st = kv4_shape(pages, kv_heads, head_dim, page, group, &sh)) return st;
  if (layers > 65535 || table_width >= (int64_t{1} << 31) || table_width * page > (int64_t{1} << 30) ||
      seqs >= (int64_t{1} << 24) / beams)
    return QMM_ERANGE;
  if (!aligned(cache, 16) || !aligned(page_table, 4) || !aligned(context, 4) || !aligned(tails, 4) ||
      !aligned(parents, 8) || !aligned(table_out, 4) || !aligned(context_out, 4))
    return QMM_EALIGN;
  Reorder a{};
  a.cache = cache;
  a.sh = sh;
  a.table = page_table;
  a.width = static_cast<int32_t>(table_width);
  a.context = context;
  a.tails = tails;
  a.parents = parents;
  a.beams = static_cast<int32_t>(beams);
  a.table_out = table_out;
  a.context_out = context_out;
  const dim3 grid(static_cast<unsigned>(seqs * beams), static_cast<unsigned>(layers),
                  static_cast<unsigned>(ceil_div(kv_heads, kReorderHeads)));
  if (static_cast<int64_t>(grid.x) * grid.y * grid.z >= (int64_t{1} << 24)) return QMM_ERANGE;
  kv4_beam_reorder_kernel<<<grid, 256, 0, as_stream(stream)>>>(a);
  return launch_status();
}
