/*
 * pa_tree.h -- attention for drafted tokens over a paged KV cache: the pass
 * that verifies a tree of drafts (or a chain of them, or runs one plain decode
 * step) against the fp16 cache of pa.h or the 8-bit cache of pa_cache.h. The
 * reference pages name a mask type for speculative decoding without describing
 * it; this call states the tree itself instead of a mask tensor.
 *
 * For sequence b with q_b current tokens, whose keys and values sit at the
 * cache positions L_b - q_b .. L_b - 1, token i attends
 *   every position below L_b - q_b,
 *   itself, and
 *   with parents     its ancestors: parents[i], parents[parents[i]], ...
 *   without parents  every current token before it (a chain)
 * out = softmax(scale * <q, K_j>) V_j over those, heads grouped as in pa.h.
 * Keys and values that a row does not attend have no effect on it, whatever
 * they hold (NaN and infinities included). A slot of the 8-bit cache that nothing
 * was written into (zero codes, zero exponent byte) is a row of zeros.
 *
 * Scores, softmax sums and outputs are accumulated in fp32, the 8-bit cache's codes and
 * exponents enter them exactly; the weights are rounded to fp16 for their product
 * with V. However long a context, no fp32 sum is of more than 65536 keys before it is
 * rounded to nearest into the next (the tensor cores' additions cut off, less than 2^-12 of
 * sum p |v| in as many). The same batch gives the same bits every time; a
 * sequence in another batch may differ in its last bits, as the work is divided
 * otherwise.
 */
#ifndef PA_TREE_H
#define PA_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A parent that is not -1 or an earlier token of its sequence: the token is
 * taken as a root and the bit is set in the status word (pa_status_read returns
 * PA_ERR_INVALID_ARG). */
#define PA_STATUS_BIT_TREE 32u
/* Most current tokens of a sequence when parents are given. */
#define PA_TREE_MAX_TOKENS 256

/*
 * pa_tree_workspace -- bytes of workspace that pa_tree_forward needs for this
 * configuration, whatever the lengths (host only).
 */
pa_status pa_tree_workspace(const pa_config* cfg, size_t* workspace_bytes);

/*
 * pa_tree_forward -- asynchronous, allocates nothing, reads the lengths on the
 * device only (so that it may be captured once and replayed as they change).
 *
 * cfg            as in pa.h, with mask_type = PA_MASK_NONE, chunk_blocks = 0 and
 *                0 < num_sms <= 65535. With parents max_seqlen_q <= PA_TREE_MAX_TOKENS.
 * tokens         rows of query and out (sum q_b, or more: the rows behind the
 *                last sequence are neither read nor written; with fewer the rows
 *                past them are left out, and PA_STATUS_BIT_PLAN says so)
 * query          device fp16 [tokens, H, hk], 16-byte aligned
 * key_cache, value_cache  fp16 as in pa.h, or e4m3 codes as in pa_cache.h; two
 *                different caches
 * key_exps, value_exps    NULL for the fp16 cache, else as in pa_cache.h
 * block_tables   device int32 [batch, max_blocks_per_seq]
 * context_lens   device int32 [batch], L_b counting the current tokens, at most
 *                max_blocks_per_seq * block_size and 2^31 - 4096
 * q_seqlens      device int32 [batch], 0 <= q_b <= max_seqlen_q (0: a padding
 *                sequence), or NULL when every row is one token of its sequence (a row
 *                of L_b = 0 is then padding)
 * parents        device int32 [tokens]: -1 for a root (a child of the last
 *                token before the drafts), else the index within the
 *                sequence's current tokens of an earlier one; or NULL
 * workspace      device, >= pa_tree_workspace's bytes, 256-byte aligned; its
 *                status word zero before the first call, as in pa.h. Calls
 *                whose work overlaps on the GPU need a workspace each.
 * out            device fp16 [tokens, H, hv], 16-byte aligned, not the query
 *
 * The lengths, the block tables and the parents must not change while the call's
 * work runs. A length that breaks a constraint (PA_STATUS_BIT_PLAN) leaves its sequence
 * out; the other sequences' rows lie where the stated lengths put them (a negative one
 * counts as 0). A block table entry outside [0, num_blocks) is never dereferenced and
 * makes the outputs of its sequence undefined (PA_STATUS_BIT_BLOCK_INDEX).
 */
pa_status pa_tree_forward(const pa_config* cfg, int64_t tokens, const void* query,
                          const void* key_cache, const void* value_cache, const uint8_t* key_exps,
                          const uint8_t* value_exps, const int32_t* block_tables,
                          const int32_t* context_lens, const int32_t* q_seqlens,
                          const int32_t* parents, void* workspace, size_t workspace_bytes,
                          void* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_TREE_H */
