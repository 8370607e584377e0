/* qmm_blocks.h -- libqmm's calls of a decode step in the form that a binding
 * calls them (the calls themselves: qmm.h). */
#ifndef QMM_BLOCKS_H_
#define QMM_BLOCKS_H_

#include "qmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * The calls of a decode step with their arguments in one block: <name>_block
 * is <name> of the words' values, one 8-byte word an argument in its order,
 * pointers and integers as int64_t, floating-point ones as double (8-byte
 * aligned; QMM_EINVAL for NULL).  For bindings that pay for each argument of a
 * foreign call, as the Python one does: 3.8 us for the 27 of kv4_attention,
 * 0.7 us for a block.
 * ------------------------------------------------------------------------- */
int kv4_append_block(const void* words);
int kv4_read_block(const void* words);
int kv4_copy_pages_block(const void* words);
int kv4_attention_block(const void* words);
int qk_norm_rope_block(const void* words);

#ifdef __cplusplus
}
#endif

#endif /* QMM_BLOCKS_H_ */
