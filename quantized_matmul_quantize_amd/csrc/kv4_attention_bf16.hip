// kv4_attention_bf16.hip -- the attention kernels for bf16 queries.

#include "kv4_attention_launch.h"

void qmm::attention_bf16(const AttnArgs& a, const AttnPlan& p, hipStream_t s) { launch_attention<QMM_BF16>(a, p, s); }
