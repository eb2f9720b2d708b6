/*
 * pa_window.h -- attention with a sliding window and a few first tokens that stay
 * visible (sinks), over the fp16 cache of pa.h or the 8-bit cache of pa_cache.h: decode
 * steps, chains of drafted tokens, whole prompts and parts of prompts. The reference
 * pages have no counterpart.
 *
 * For sequence b with q_b current tokens, whose keys and values sit at the cache
 * positions L_b - q_b .. L_b - 1, the token at position p attends position j <= p where
 *   j > p - window   or   j < sinks
 * out = softmax(scale * <q, K_j>) V_j over those, heads grouped as in pa.h. Every row sees
 * itself. With window >= L_b this is causal attention. Keys and values that a row does not
 * attend have no effect on it, whatever they hold (NaN and infinities included), and a
 * block none of whose positions is attended is not looked at: its table entry may be
 * anything (pa_blocks.h leaves -1 where it gave a block back).
 *
 * Precision, and what holds of equal batches, are pa_tree_forward's.
 */
#ifndef PA_WINDOW_H
#define PA_WINDOW_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   window  keys that a token attends, itself among them; > 0
 *   sinks   first positions of a sequence that stay visible; >= 0
 */
typedef struct pa_window {
  int32_t window;
  int32_t sinks;
} pa_window;

/*
 * pa_window_workspace -- bytes of workspace that pa_window_forward needs for this
 * configuration, whatever the lengths (host only).
 */
pa_status pa_window_workspace(const pa_config* cfg, const pa_window* win, size_t* workspace_bytes);

/*
 * pa_window_forward -- asynchronous, allocates nothing, reads the lengths on the
 * device only (so that it may be captured once and replayed as they change).
 *
 * cfg            as in pa.h, with mask_type = PA_MASK_NONE, chunk_blocks = 0 and
 *                0 < num_sms <= 65535
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
 * workspace      device, >= pa_window_workspace's bytes, 256-byte aligned; its
 *                status word zero before the first call, as in pa.h. Calls
 *                whose work overlaps on the GPU need a workspace each.
 * out            device fp16 [tokens, H, hv], 16-byte aligned, not the query
 *
 * The lengths and the block tables must not change while the call's work runs. A length
 * that breaks a constraint (PA_STATUS_BIT_PLAN) leaves its sequence out; the other
 * sequences' rows lie where the stated lengths put them (a negative one counts as 0). An
 * entry outside [0, num_blocks) of a block that is attended is never dereferenced and
 * makes the outputs of its sequence undefined (PA_STATUS_BIT_BLOCK_INDEX).
 */
pa_status pa_window_forward(const pa_config* cfg, const pa_window* win, int64_t tokens,
                            const void* query, const void* key_cache, const void* value_cache,
                            const uint8_t* key_exps, const uint8_t* value_exps,
                            const int32_t* block_tables, const int32_t* context_lens,
                            const int32_t* q_seqlens, void* workspace, size_t workspace_bytes,
                            void* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_WINDOW_H */
