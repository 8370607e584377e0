// kv4_prefix_bf16.hip -- the attention over shared prefixes for bf16 queries.

#include "kv4_prefix_launch.h"

void qmm::prefix_attention_bf16(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s) {
  launch_prefix<QMM_BF16>(a, prefix, own, together, s);
}
