/*
 * pa_blocks.h -- the blocks of a paged KV cache, handed out and given back on the GPU:
 * block tables and slot maps from the lengths of the requests, without a copy of the
 * lengths to the host. The reference pages have no counterpart; the tables are those of pa.h.
 *
 * A pool is five device int32 arrays of the caller's:
 *   block_tables  [batch, max_blocks_per_seq]
 *   held          [batch]: entries of the row that were handed out
 *   gone          [batch]: of those, how many behind the first ceil(sinks / bs) were given
 *                 back since, as the window moved on
 *   free_blocks   [num_blocks]: the first *count of them are free, the last one on top
 *   count         [1]
 * A fresh pool has held and gone zero and every block free. An entry that is not held
 * reads -1 in a table that started so. No block belongs to two rows.
 */
#ifndef PA_BLOCKS_H
#define PA_BLOCKS_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* More blocks were asked for than were free (pa_status_read returns
 * PA_ERR_BUFFER_TOO_SMALL), or the pool's count is not one of its blocks. */
#define PA_STATUS_BIT_POOL 64u

/*
 *   batch               0 < B <= 2048
 *   block_size          bs, a multiple of 16
 *   num_blocks          physical blocks; num_blocks * bs < 2^31
 *   max_blocks_per_seq  row length of block_tables; batch * max_blocks_per_seq < 2^31
 *   window              keys that a token attends, itself among them (pa_window.h); 0: all,
 *                       so that nothing is given back before the request ends
 *   sinks               first positions that stay visible, >= 0
 */
typedef struct pa_blocks_config {
  int32_t batch;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t window;
  int32_t sinks;
} pa_blocks_config;

/*
 * pa_blocks_step -- one step of the pool, asynchronous on the caller's stream.
 *
 * context_lens  device int32 [batch], L_b counting the current tokens; 0 ends the
 *               request of row b
 * q_seqlens     device int32 [batch], 0 <= q_b <= L_b, or NULL when every row is one token
 *               of row b (a row of L_b = 0 is then padding)
 * tokens        elements of slots and positions
 * slots         device int64 [tokens] or NULL
 * positions     device int32 [tokens] or NULL
 *
 * First, blocks are given back: those of rows with L_b = 0, and, with a window, those
 * behind the sinks' blocks whose positions no current or later token attends (all of
 * them at most L_b - q_b - window). Their entries become -1. They come to lie on the
 * stack so that the first one, in the order of rows and entries, is on top.
 * Then every row is brought up to ceil(L_b / bs) entries, the blocks taken from the top, in
 * the same order (so the blocks that a step gives back are the first that it hands
 * out, and a step that gives back what the step before handed out leaves the stack as that
 * found it). A row that holds more keeps them. Once the stack is empty the
 * rest is not handed out (PA_STATUS_BIT_POOL); held says what was, and a later step goes on
 * from there.
 * Last, token i of sequence b (row sum_{b' < b} q_b' + i) has positions = L_b - q_b + i = p and
 * slots = block_tables[b][p / bs] * bs + p % bs, or -1 where there is no block. Rows behind the
 * last sequence's get -1 in both, so that the calls of pa_cache.h leave them out.
 *
 * `status` is a device uint32 or NULL: PA_STATUS_BIT_PLAN for a row whose lengths or
 * whose held or gone break a constraint (its blocks stay as they are, its tokens get -1) and for
 * lengths that are more than `tokens` (where slots or positions are given),
 * PA_STATUS_BIT_BLOCK_INDEX for an entry outside [0, num_blocks) that is given back, handed
 * out or a current token's, PA_STATUS_BIT_POOL.
 *
 * The arrays must not change while the call's work runs; two steps of one pool must not
 * overlap.
 */
pa_status pa_blocks_step(const pa_blocks_config* cfg, const int32_t* context_lens,
                         const int32_t* q_seqlens, int32_t* block_tables, int32_t* held,
                         int32_t* gone, int32_t* free_blocks, int32_t* count, int64_t tokens,
                         int64_t* slots, int32_t* positions, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_BLOCKS_H */
