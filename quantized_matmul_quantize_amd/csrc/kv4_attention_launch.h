// kv4_attention_launch.h -- from a launch plan to the kernel that it names.
#pragma once

#include "kv4_attention.h"
#include "kv4_attention_chunk.h"

namespace qmm {
namespace {

template <int DT, int D, int GROUP>
void launch_shape(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.blocks));
  constexpr int kTiles = attention_tiles(D, GROUP);
  if (!p.ws) {
    attention_chunk_kernel<DT, D, GROUP, attention_chunk_tiles(D, GROUP)><<<grid, 256, 0, s>>>(a);
  } else if (p.pk == 2) {
    if constexpr (attention_pairs(D, GROUP)) attention_kernel<DT, D, GROUP, 2, 1><<<grid, 256, 0, s>>>(a);
  } else if (p.nt == 1) {
    attention_kernel<DT, D, GROUP, 1, 1><<<grid, 256, 0, s>>>(a);
  } else {
    attention_kernel<DT, D, GROUP, 1, kTiles><<<grid, 256, 0, s>>>(a);
  }
}

template <int DT>
void launch_attention(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int D = a.sh.D, g = a.sh.group;
  if (D == 64) {
    if (g == 32) launch_shape<DT, 64, 32>(a, p, s);
    else launch_shape<DT, 64, 64>(a, p, s);
  } else if (D == 128) {
    if (g == 32) launch_shape<DT, 128, 32>(a, p, s);
    else if (g == 64) launch_shape<DT, 128, 64>(a, p, s);
    else launch_shape<DT, 128, 128>(a, p, s);
  } else {
    if (g == 32) launch_shape<DT, 256, 32>(a, p, s);
    else if (g == 64) launch_shape<DT, 256, 64>(a, p, s);
    else launch_shape<DT, 256, 128>(a, p, s);
  }
  if (p.splits > 1) {
    const dim3 grid(static_cast<unsigned>(p.max_q < 1024 ? p.max_q : 1024), static_cast<unsigned>(a.q_heads),
                    static_cast<unsigned>(a.seqs));
    const int rows = static_cast<int>(p.rows);
    if (D == 64) attention_join_kernel<DT, 64><<<grid, 256, 0, s>>>(a, rows);
    else if (D == 128) attention_join_kernel<DT, 128><<<grid, 256, 0, s>>>(a, rows);
    else attention_join_kernel<DT, 256><<<grid, 256, 0, s>>>(a, rows);
  }
}

}  // namespace
}  // namespace qmm
