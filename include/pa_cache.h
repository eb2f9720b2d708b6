/*
 * pa_cache.h -- what surrounds the attention of pa.h in a serving step: the
 * norms and the rotation of queries and keys, and a paged KV cache held in 8
 * bits, written and read back. The reference pages have no counterpart; the
 * caches are addressed as pa.h addresses its own (block tables, context
 * lengths that count the current tokens, token-concatenated rows).
 *
 * The 8-bit cache
 * ---------------
 *   key_cache    e4m3 codes [num_blocks, bs, Hk, hk] (the layout of pa.h's fp16
 *                cache), 16-byte aligned
 *   key_exps     uint8      [num_blocks, Hk, bs]: one power-of-two exponent per
 *                token and kv head, biased by 127; 16-byte aligned
 *   value_cache, value_exps the same with hv
 * For one row x of a (token, kv head): e is the least integer >= -32 with
 * max |x| <= 448 * 2^e, the maximum over the finite elements (-32 when that is
 * 0); element d is held as RN_e4m3(x_d * 2^-e), a non-finite one as NaN; the
 * exponent byte is e + 127. It stands for code * 2^e. With a power of two the
 * scaling itself is exact, so an element is off by at most half a step of
 * e4m3 (2^-4 relative, 2^-10 * 2^e absolute below 2^-6 * 2^e).
 *
 * Conventions are those of pa.h: every function returns a pa_status, is
 * asynchronous on the caller's stream, allocates nothing, and returns host-side
 * errors before anything is enqueued. `status` is a device uint32 or NULL; the
 * kernels only OR bits into it (pa_status_read takes its address; it returns
 * PA_ERR_INVALID_ARG for the PLAN and POSITION bits):
 *   PA_STATUS_BIT_BLOCK_INDEX  a block table entry outside [0, num_blocks); the
 *                              tokens of that block are neither stored nor read
 *   PA_STATUS_BIT_PLAN         a length breaks a constraint; that sequence (or
 *                              the rows past `tokens`) is left out. The other
 *                              sequences' rows lie where the stated lengths put
 *                              them (a negative one counts as 0). A call of
 *                              no tokens looks at none
 *   PA_STATUS_BIT_POSITION     a position outside [-1, max_positions); that
 *                              token is left out
 *   PA_STATUS_BIT_WORKSPACE    an output row outside [0, out_rows); left out
 * What is left out keeps the bytes it had: so do rows behind the last
 * sequence and cache slots that no token of the call names.
 */
#ifndef PA_CACHE_H
#define PA_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "pa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_STATUS_BIT_POSITION 16u

/*
 * Norm and rotation of the query and key heads.
 *
 * For a head row x of hk dims: y = x * rsqrt(mean(x^2) + eps) * weight when its
 * weight is given (else y = x), then the first rotary_dim dims of y are turned
 * in pairs (a, b) -> (a c - b s, b c + a s) with c = cos_sin[p][i] and
 * s = cos_sin[p][rotary_dim / 2 + i] for pair i at position p: dims
 * (i, i + rotary_dim / 2), or (2i, 2i + 1) when interleaved. fp32 throughout,
 * rounded once.
 *
 *   num_heads, kv_heads  H, Hk > 0 (no divisibility asked here)
 *   head_size            hk in (0, 576], a multiple of 16
 *   rotary_dim           in [0, hk], a multiple of 16
 *   max_positions        rows of cos_sin, > 0
 *   eps                  >= 0
 */
typedef struct pa_rotary {
  int32_t num_heads;
  int32_t kv_heads;
  int32_t head_size;
  int32_t rotary_dim;
  int32_t interleaved;
  int32_t max_positions;
  float eps;
} pa_rotary;

/*
 * pa_qk_norm_rope -- norm and rotate the heads of `tokens` tokens, in one pass.
 *
 * query, key          fp16; head h of token t at [t * stride + h * hk], so that
 *                     both may point into one packed projection; strides in
 *                     elements, multiples of 8 and at least H * hk (Hk * hk);
 *                     16-byte aligned
 * q_weight, k_weight  fp16 [hk], 16-byte aligned, each may be NULL (no norm)
 * cos_sin             fp32 [max_positions, rotary_dim], 16-byte aligned (may be
 *                     NULL when rotary_dim is 0)
 * positions           int32 [tokens]; -1 marks a padding token, left out
 * q_out, k_out        fp16 [tokens, H, hk], [tokens, Hk, hk], 16-byte aligned.
 *                     q_out may be query itself when it is dense (stride =
 *                     H * hk), and k_out key; no other overlap.
 */
pa_status pa_qk_norm_rope(const pa_rotary* rot, int64_t tokens, const void* query,
                          int64_t query_stride, const void* key, int64_t key_stride,
                          const void* q_weight, const void* k_weight, const float* cos_sin,
                          const int32_t* positions, void* q_out, void* k_out, uint32_t* status,
                          void* stream);

/*
 * Positions of several axes, as tokens of images and video have them (time, height,
 * width): pair i of the rotation turns by the position of one of them.
 *
 *   count     axes, 1 to PA_MAX_AXES
 *   cyclic    0: the first sections[0] pairs turn by axis 0, the next sections[1] by
 *             axis 1, and so on. Else pair i turns by axis a = i % count where a > 0 and
 *             i < count * sections[a], and by axis 0 otherwise
 *   sections  pairs of each axis, >= 0, together rotary_dim / 2; cyclic: each axis but
 *             the first finds its places, count * (sections[a] - 1) + a < rotary_dim / 2
 */
#define PA_MAX_AXES 4
typedef struct pa_axes {
  int32_t count;
  int32_t cyclic;
  int32_t sections[PA_MAX_AXES];
} pa_axes;

/*
 * pa_qk_norm_rope_axes -- pa_qk_norm_rope with positions int32 [axes->count][tokens].
 * A token one of whose positions is -1 is left out as padding; one outside [-1,
 * max_positions) sets the POSITION bit and leaves its token out. Tokens whose
 * positions are the same on every axis get the bits that pa_qk_norm_rope gives.
 */
pa_status pa_qk_norm_rope_axes(const pa_rotary* rot, const pa_axes* axes, int64_t tokens,
                               const void* query, int64_t query_stride, const void* key,
                               int64_t key_stride, const void* q_weight, const void* k_weight,
                               const float* cos_sin, const int32_t* positions, void* q_out,
                               void* k_out, uint32_t* status, void* stream);

/*
 * The 8-bit cache and a batch over it.
 *
 *   batch               0 < B <= 2048
 *   kv_heads            Hk > 0
 *   head_size_k/_v      hk, hv in (0, 576], multiples of 16
 *   block_size          bs, a multiple of 16
 *   num_blocks          physical blocks; num_blocks * bs < 2^31
 *   max_blocks_per_seq  row length of block_tables
 *   max_rows            pa_cache_write/_store: the largest q_b; pa_cache_read:
 *                       the largest context_lens[b] - starts[b]; >= 0
 */
typedef struct pa_cache_config {
  int32_t batch;
  int32_t kv_heads;
  int32_t head_size_k;
  int32_t head_size_v;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t max_rows;
} pa_cache_config;

/*
 * pa_cache_write -- quantise the current tokens' keys and values into the cache.
 *
 * Token i of sequence b (row sum_{b' < b} q_b' + i of key and value) goes to
 * cache position context_lens[b] - q_b + i. Sequences with q_b = 0 are padding.
 *
 * tokens        rows of key and value; rows past sum q_b are not read
 * key, value    fp16, as in pa_qk_norm_rope (strides in elements)
 * q_seqlens     device int32 [batch], or NULL when every row is one token of its
 *               sequence (a row of context_lens[b] = 0 is then padding)
 * No two current tokens may name the same cache slot (a block that two
 * sequences share must be copied before one of them writes into it); a slot
 * that is named twice ends up holding bytes of either row.
 */
pa_status pa_cache_write(const pa_cache_config* cfg, int64_t tokens, const void* key,
                         int64_t key_stride, const void* value, int64_t value_stride,
                         const int32_t* block_tables, const int32_t* context_lens,
                         const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps,
                         void* value_cache, uint8_t* value_exps, uint32_t* status, void* stream);

/*
 * pa_cache_store -- pa_qk_norm_rope and pa_cache_write in one pass: the
 * queries are normed, rotated and written to q_out, the keys are normed,
 * rotated and quantised (from fp32, without a rounding to fp16 between) into
 * the cache, the values are quantised into the cache.
 *
 * rot->kv_heads = cfg->kv_heads and rot->head_size = cfg->head_size_k.
 * positions may be NULL: a token's position is then its cache position. A
 * token of position -1 is left out altogether.
 */
pa_status pa_cache_store(const pa_cache_config* cfg, const pa_rotary* rot, int64_t tokens,
                         const void* query, int64_t query_stride, const void* key,
                         int64_t key_stride, const void* value, int64_t value_stride,
                         const void* q_weight, const void* k_weight, const float* cos_sin,
                         const int32_t* positions, const int32_t* block_tables,
                         const int32_t* context_lens, const int32_t* q_seqlens, void* key_cache,
                         uint8_t* key_exps, void* value_cache, uint8_t* value_exps, void* q_out,
                         uint32_t* status, void* stream);

/*
 * pa_cache_store_axes -- pa_cache_store with positions int32 [axes->count][tokens], as in
 * pa_qk_norm_rope_axes (not NULL; where a token is stored goes by the lengths alone).
 */
pa_status pa_cache_store_axes(const pa_cache_config* cfg, const pa_rotary* rot,
                              const pa_axes* axes, int64_t tokens, const void* query,
                              int64_t query_stride, const void* key, int64_t key_stride,
                              const void* value, int64_t value_stride, const void* q_weight,
                              const void* k_weight, const float* cos_sin,
                              const int32_t* positions, const int32_t* block_tables,
                              const int32_t* context_lens, const int32_t* q_seqlens,
                              void* key_cache, uint8_t* key_exps, void* value_cache,
                              uint8_t* value_exps, void* q_out, uint32_t* status, void* stream);

/*
 * pa_cache_read -- read cached tokens back as fp16 rows.
 *
 * Position starts[b] + i of sequence b, up to context_lens[b], is written to
 * row out_starts[b] + i of k_out and v_out (a value beyond fp16's range as an
 * infinity). With out_starts at multiples of the block size the outputs are
 * themselves caches that pa_forward reads.
 *
 * starts      device int32 [batch], or NULL for zeros
 * out_starts  device int32 [batch]
 * k_out       fp16 [out_rows, Hk, hk], 16-byte aligned; v_out the same with hv
 */
pa_status pa_cache_read(const pa_cache_config* cfg, const void* key_cache, const uint8_t* key_exps,
                        const void* value_cache, const uint8_t* value_exps,
                        const int32_t* block_tables, const int32_t* starts,
                        const int32_t* context_lens, const int32_t* out_starts, int64_t out_rows,
                        void* k_out, void* v_out, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_CACHE_H */
