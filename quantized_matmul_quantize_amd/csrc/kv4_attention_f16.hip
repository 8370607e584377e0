// kv4_attention_f16.hip -- the attention kernels for binary16 queries.

#include "kv4_attention_launch.h"

void qmm::attention_f16(const AttnArgs& a, const AttnPlan& p, hipStream_t s) { launch_attention<QMM_F16>(a, p, s); }
