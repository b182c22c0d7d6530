/*
 * kv4.h — C ABI of a paged cache of keys and values in 4 bits, for serving: new
 * tokens are written to it with the position rotation applied on the way, rows are
 * read back, and attention runs over it. Part of liblora_nf4.so. A decoded token's
 * path through a layer is
 *     rmsnorm_fwd_quant -> w4_matvec_multi (q, k, v) -> kv4_append -> kv4_attention
 *     -> w4_matvec
 * (norm_w4.h). The pages keep the cache in blocks of tokens reached through a table
 * ("Unsloth in three lines of code", sections 1 and 2).
 *
 * Conventions as in lora_nf4.h: device pointers owned by the caller (16-byte
 * aligned, workspaces 256-byte), bf16 as uint16_t bit patterns, work enqueued on
 * `stream` of the current device, nothing allocated or synchronized, arguments
 * checked on the host before any HIP call (ln_status codes), outputs disjoint from
 * inputs and from each other (LN_EALIAS), no state kept between calls.
 * Floating-point inputs must be finite (not checked). Whole numbers that lie in
 * device memory (slots, positions, page numbers, lengths) cannot be checked without
 * a synchronization; the kernels check them against the sizes of what they index,
 * and each entry point says what a number out of range does. Nothing outside the
 * operands is ever read or written.
 *
 * The cache of one layer: n_pages pages of page_size tokens, n_kv heads of head_dim
 * values, a step and a least value per token, head and `group` values:
 *     x = lo + s c,   c in 0 .. 15
 *   k_codes   uint8 [n_pages][n_kv][page_size][head_dim / 2]; byte
 *             g head_dim / 8 + 4 c + b of a row holds element 32 c + 8 g + b in its
 *             low nibble and element 32 c + 8 g + b + 4 in its high one (g, b in
 *             0 .. 3, c < head_dim / 32)
 *   v_codes   uint8 [n_pages][n_kv][page_size / 4][2 head_dim]; byte
 *             r head_dim / 8 + 4 c + i of four tokens holds, for token i of them,
 *             element 32 c + 2 r in its low nibble and the next in its high one
 *             (r in 0 .. 15)
 *   k_scales, v_scales   bf16 [n_pages][n_kv][head_dim / group][page_size][2]: (s, lo)
 * Slot t is token t % page_size of page t / page_size. Both orders make what one
 * lane of the attention reads consecutive; a token's bytes are its own in both, so
 * that tokens are written independently of each other.
 *   head_dim  64, 128 or 256;  group 32, 64 or 128, dividing head_dim
 *   page_size a multiple of 32 up to LN_KV4_MAX_PAGE
 *   n_pages   1 .. 2^31 - 1, n_pages page_size < 2^40;  n_kv 1 .. LN_KV4_MAX_HEADS
 */
#ifndef KV4_H
#define KV4_H

#include <stddef.h>
#include <stdint.h>

#include "lora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LN_KV4_MAX_PAGE 4096
#define LN_KV4_MAX_HEADS 1024 /* of queries, and of keys */

typedef struct {
    int64_t n_pages;
    int32_t page_size, n_kv, head_dim, group;
    uint8_t* k_codes;
    uint16_t* k_scales;
    uint8_t* v_codes;
    uint16_t* v_scales;
} ln_kv4_cache;

/*
 * kv4_append — T tokens' queries and keys rotated, keys and values written to the cache:
 *     for each pair of a head's first rot_dim elements, angle i of the token's position,
 *     x1' = x1 cos_i - x2 sin_i,   x2' = x2 cos_i + x1 sin_i
 * (the sums in float64, rounded to float32 and then to bf16; elements from rot_dim on
 * rounded to bf16), and for each group of `group` bf16 elements of a key or value
 *     lo = min x,   s = bf16(f32(f32(max x - lo) / 15)),
 *     c = min(15, nearest integer to f32(x - lo) / s, halves to even; 0 where s = 0)
 * (max x - lo must be finite in float32).
 *   dtype       LN_BF16 or LN_F32, of q, k and v
 *   q, k, v     [T] rows of n_q, n_kv and n_kv heads, each row contiguous and q_stride,
 *               k_stride, v_stride elements after the one before (for parts of one wider
 *               matrix; multiples of 16 bytes, at least a row). q may be NULL together with q_out
 *   cos, sin    float32 [n_pos][rot_dim / 2], or both NULL with rot_dim 0: no rotation
 *   rot_dim     a multiple of 16 up to head_dim
 *   interleaved 0: pairs (i, i + rot_dim / 2);  1: pairs (2 i, 2 i + 1)
 *   positions   int64 [T], rows of cos and sin (NULL without rotation). A position out of
 *               range leaves the token out of the cache and zeros in its row of q_out
 *   slots       int64 [T]. A slot out of range (-1, say) leaves the token out of the cache.
 *               Where several tokens have the same slot the last one is kept
 *   q_out       bf16 [T][n_q head_dim], contiguous (output)
 *   cache       HOST struct, read during the call only; slots not named keep what they hold
 * n_q up to LN_KV4_MAX_HEADS. T >= 0 (0: nothing to do, token operands may be NULL), T < 2^24.
 */
int kv4_append(int64_t T, int32_t n_q, int dtype, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
               const void* v, int64_t v_stride, const float* cos, const float* sin, int64_t n_pos, int32_t rot_dim,
               int32_t interleaved, const int64_t* positions, const int64_t* slots, uint16_t* q_out,
               const ln_kv4_cache* cache, void* stream);

/*
 * kv4_read — the keys and values of T slots as rows: f32(s c + lo), rounded once more for
 * LN_BF16.
 *   slots     int64 [T], in any order; one out of range gives rows of zeros
 *   k, v      [T][n_kv head_dim] of out_dtype (outputs; either may be NULL)
 * T >= 0, T < 2^24.
 */
int kv4_read(int64_t T, const int64_t* slots, const ln_kv4_cache* cache, int out_dtype, void* k, void* v,
             void* stream);

/*
 * kv4_attention — attention of B sequences over their keys and values in the cache. Sequence
 * b has lens[b] keys, key t in slot t % page_size of page block_table[b][t / page_size], and
 * its queries stand for the last n_b of them: query j sees the keys
 *     t <= lens[b] - n_b + j,   and with a window  t > lens[b] - n_b + j - window
 *     y = sum_t p_t v_t,   p = softmax_t(scale q k_t),   lse = ln sum_t exp(scale q k_t)
 * Query head i reads key head i / (n_q / n_kv). A query that sees no key (an empty sequence,
 * more queries than keys) gives y = 0 and lse = -infinity. Products of q (bf16) with codes
 * and all sums are float32; p_t s_t is rounded to bf16 before it multiplies c_t - 8 (off by at
 * most 2^-8 p_t s_t |c_t - 8| a key); y is rounded once. p_t stands there for a weight below 2^8 that is
 * divided by the weights' sum at the end, so scale log2 e q k_t and 2^8 sum_t |v_t| must be finite in float32.
 *   q           bf16 [T] rows of n_q heads, q_stride elements apart (a multiple of 8, at least
 *               a row)
 *   cu_q        int32 [B + 1]: sequence b has rows cu_q[b] .. cu_q[b + 1] - 1 (clamped to
 *               0 .. T). NULL: one query each, row b (then T = B)
 *   max_q       an upper bound of n_b, or 0 if none is known (rows past it may be left as they
 *               were). Taken as 1 where cu_q is NULL, also by the size of the workspace
 *   lens        int32 [B] (clamped to 0 .. max_pages page_size)
 *   block_table int32 [B][max_pages]. A page out of range has no keys
 *   window      0: none
 *   scale       > 0, scale log2 e finite in float32
 *   y           bf16 [T][n_q head_dim] contiguous;  lse  float32 [T][n_q] or NULL (outputs).
 *               Rows of no sequence are left as they were
 *   workspace   kv4_attention_workspace_bytes(...) bytes, where a sequence's keys are split
 *               over workgroups (float32 sums of the parts, joined in a fixed order: the result
 *               does not depend on the run); two calls that may run at the same time need
 *               one each
 * n_q a multiple of n_kv, up to LN_KV4_MAX_HEADS. 0 <= T < 2^24, T n_q <= 2^30, 1 <= B < 2^20,
 * max_pages >= 1, max_pages page_size <= 2^30, and row blocks of 16 times tiles of 32 keys,
 * (T n_q / n_kv / 16 + B) (max_pages page_size / 32 + 2), fewer than 2^36.
 */
int kv4_attention(int64_t T, int64_t B, int32_t n_q, const uint16_t* q, int64_t q_stride, const int32_t* cu_q,
                  int32_t max_q, const int32_t* lens, const int32_t* block_table, int64_t max_pages, int32_t window,
                  float scale, const ln_kv4_cache* cache, uint16_t* y, float* lse, void* workspace,
                  size_t workspace_bytes, void* stream);

/* Workspace bytes kv4_attention needs (0 if the sizes are invalid or T = 0). */
size_t kv4_attention_workspace_bytes(int64_t T, int64_t B, int32_t n_q, int32_t n_kv, int32_t head_dim,
                                     int32_t max_q, int64_t max_pages, int32_t page_size);

#ifdef __cplusplus
}
#endif

#endif /* KV4_H */
