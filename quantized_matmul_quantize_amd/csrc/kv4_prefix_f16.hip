// kv4_prefix_f16.hip -- the attention over shared prefixes for binary16 queries.

#include "kv4_prefix_launch.h"

void qmm::prefix_attention_f16(const SharedArgs& a, const AttnPlan& prefix, const AttnPlan& own, bool together, hipStream_t s) {
  launch_prefix<QMM_F16>(a, prefix, own, together, s);
}
