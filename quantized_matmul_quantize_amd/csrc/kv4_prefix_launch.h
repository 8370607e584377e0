// kv4_prefix_launch.h -- from the plans of a batch with shared prefixes to the
// kernels that they name.
#pragma once

#include "kv4_attention.h"
#include "kv4_attention_chunk.h"
#include "kv4_attention_rows.h"

namespace qmm {
namespace {

template <int DT, int D, int GROUP, int PK, int NT, Part PART>
__global__ __launch_bounds__(256, attention_occupancy(D, GROUP, PK, NT)) void attention_part_kernel(SharedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * Shape<D, GROUP, PK, NT>::kWaveBytes];
  attention_block<DT, D, GROUP, PK, NT, PART>(a, blockIdx.x, lds);
}
// (types of their own: the host's pass compiles no device function for two kernels)
template <int NT>
struct BothArgs : SharedArgs {
  uint32_t prefix_blocks;
};
template <int DT, int D, int GROUP, int PK, int NT>
__global__ __launch_bounds__(256, attention_occupancy(D, GROUP, PK, NT)) void attention_both_kernel(BothArgs<NT> a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * Shape<D, GROUP, PK, NT>::kWaveBytes];
  static_assert(Shape<D, GROUP, PK, 1>::kWaveBytes <= Shape<D, GROUP, PK, NT>::kWaveBytes, "the own parts' memory");
  if (blockIdx.x < a.prefix_blocks) attention_block<DT, D, GROUP, PK, NT, kPrefix>(a, blockIdx.x, lds);
  else attention_block<DT, D, GROUP, PK, 1, kOwn>(a, blockIdx.x - a.prefix_blocks, lds);
}
template <int DT, int D, int GROUP, int NT>
__global__ __launch_bounds__(256, D / GROUP < 8 ? 2 : 1) void attention_own_chunk_kernel(SharedArgs a) {
  using L = Chunk<D, GROUP, NT>;
  __shared__ __attribute__((aligned(16))) uint8_t keys[2 * L::kKBuffer], values[2 * L::kVBuffer];
  attention_chunk_block<DT, D, GROUP, NT, kOwn>(a, blockIdx.x, keys, values);
}

template <int DT, int D, int GROUP, Part PART>
void launch_part(const SharedArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.blocks));
  constexpr int kTiles = attention_tiles(D, GROUP);
  if (!p.ws) {
    if constexpr (PART == kPrefix) attention_rows_kernel<DT, D, GROUP><<<grid, Rows<DT, D, GROUP>::kThreads, 0, s>>>(a);
    else attention_own_chunk_kernel<DT, D, GROUP, attention_chunk_tiles(D, GROUP)><<<grid, 256, 0, s>>>(a);
  } else if (p.pk == 2) {
    // (a prefix of up to 8 rows has own parts of as few: both are in one launch)
    if constexpr (PART == kOwn && attention_pairs(D, GROUP)) attention_part_kernel<DT, D, GROUP, 2, 1, PART><<<grid, 256, 0, s>>>(a);
  } else if (p.nt == 1) {
    attention_part_kernel<DT, D, GROUP, 1, 1, PART><<<grid, 256, 0, s>>>(a);
  } else {
    attention_part_kernel<DT, D, GROUP, 1, kTiles, PART><<<grid, 256, 0, s>>>(a);
  }
}
template <int DT, int D, int GROUP>
void launch_parts(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s) {
  if (together) {
    const dim3 grid(static_cast<unsigned>(prefix.blocks + own.blocks));
    const uint32_t first = static_cast<uint32_t>(prefix.blocks);
    constexpr int kTiles = attention_tiles(D, GROUP);
    if (prefix.pk == 2) {
      if constexpr (attention_pairs(D, GROUP)) attention_both_kernel<DT, D, GROUP, 2, 1><<<grid, 256, 0, s>>>({a, first});
    } else if (prefix.nt == 1) {
      attention_both_kernel<DT, D, GROUP, 1, 1><<<grid, 256, 0, s>>>({a, first});
    } else {
      attention_both_kernel<DT, D, GROUP, 1, kTiles><<<grid, 256, 0, s>>>({a, first});
    }
    return;
  }
  launch_part<DT, D, GROUP, kPrefix>(a, prefix, s);
  launch_part<DT, D, GROUP, kOwn>(a, own, s);
}

template <int DT>
void launch_prefix(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s) {
  const int D = a.sh.D, g = a.sh.group;
  if (D == 64) {
    if (g == 32) launch_parts<DT, 64, 32>(a, prefix, own, together, s);
    else launch_parts<DT, 64, 64>(a, prefix, own, together, s);
  } else if (D == 128) {
    if (g == 32) launch_parts<DT, 128, 32>(a, prefix, own, together, s);
    else if (g == 64) launch_parts<DT, 128, 64>(a, prefix, own, together, s);
    else launch_parts<DT, 128, 128>(a, prefix, own, together, s);
  } else {
    if (g == 32) launch_parts<DT, 256, 32>(a, prefix, own, together, s);
    else if (g == 64) launch_parts<DT, 256, 64>(a, prefix, own, together, s);
    else launch_parts<DT, 256, 128>(a, prefix, own, together, s);
  }
  const unsigned queries = static_cast<unsigned>(own.max_q < 1024 ? own.max_q : 1024), seqs = static_cast<unsigned>(a.seqs);
  if (static_cast<int64_t>(a.T) * a.q_heads >= 8 * device_cus()) {
    const dim3 grid(queries, static_cast<unsigned>(ceil_div(a.q_heads, kWaves)), seqs);
    if (D == 64) attention_join_rows_kernel<DT, 64><<<grid, 256, 0, s>>>(a);
    else if (D == 128) attention_join_rows_kernel<DT, 128><<<grid, 256, 0, s>>>(a);
    else attention_join_rows_kernel<DT, 256><<<grid, 256, 0, s>>>(a);
  } else {
    const dim3 grid(queries, static_cast<unsigned>(a.q_heads), seqs);
    if (D == 64) attention_join_parts_kernel<DT, 64><<<grid, 256, 0, s>>>(a);
    else if (D == 128) attention_join_parts_kernel<DT, 128><<<grid, 256, 0, s>>>(a);
    else attention_join_parts_kernel<DT, 256><<<grid, 256, 0, s>>>(a);
  }
}

}  // namespace
}  // namespace qmm
