/*
 * fp8bs_serve.h -- operators of a serving step of libfp8bs.so (gfx950) around
 * the attention of fp8bs_attn.h and the GEMMs of fp8bs.h: the latent vectors
 * quantized as they are written into the paged cache and read back, the
 * absorbed attention over a cache held in 4 bits, a whole mixture-of-experts
 * layer for a few tokens, and log probabilities with entropy and alternatives
 * (and their gradient).
 *
 * Conventions as in fp8bs_attn.h: device pointers to caller-owned memory, work
 * enqueued on `stream` without synchronizing, arguments checked on the host
 * before anything is enqueued, an fp8bs_status returned. The library allocates
 * nothing; workspaces are the caller's, sized by the *_workspace_bytes
 * functions, their contents on entry do not matter; calls that may run at the
 * same time need their own. Every entry point can be captured into a HIP graph
 * and gives the same bits for the same inputs. Sizes whose launch would pass
 * 2^32 - 1 threads are refused (FP8BS_ERR_TOO_LARGE). Pointers are 16-byte
 * aligned unless said otherwise; int32 and float32 side arrays (offsets,
 * lengths, tables, expert ids and weights, lse, norm and so on) 4-byte.
 */
#ifndef FP8BS_SERVE_H
#define FP8BS_SERVE_H

#include "fp8bs_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BS_SERVE_VERSION 1

/*
 * A further kind of paged cache beside those of enum fp8bs_cache, 400 bytes a
 * token: the 512 latent numbers as E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives; bit 3 is the sign), groups of 32 sharing a power of two.
 *   cache        uint8 [pages][page][256]: column 2i in the lower half of byte
 *                i, column 2i + 1 in the upper half
 *   cache_scales uint8 [pages][page][16]: byte 127 + e says 2^e; 1 .. 254
 *   cache_rope   BF16 [pages][page][64]: the rotary numbers
 */
#define FP8BS_CACHE_FP4 2

/*
 * The newest tokens of B requests into their pages: request b's cu[b] ..
 * cu[b+1]-1 of the packed rows are its tokens at positions lens[b] - n ..
 * lens[b] - 1, n of them, lens[b] being its length with them.
 *   latent [T][512] BF16, latent_stride numbers from token to token
 *   rope   [T][64]  BF16, rope_stride numbers from token to token
 *   cu     [B+1] int32: non-decreasing, within [0, T] (precondition; the
 *          kernel stays within the T rows); rows outside cu[0] .. cu[B]-1 are
 *          not used
 *   table  [B][table_width] int32, lens [B] int32 as for fp8bs_mla_decode
 * What is written, by cache_kind:
 *   FP8BS_CACHE_BF16  cache BF16 [pages][page][576], a copy (cache_scales and
 *                     cache_rope unused, NULL)
 *   FP8BS_CACHE_FP8   cache uint8 [pages][page][512], cache_scales float32
 *                     [pages][page][4], cache_rope: codes and scales as
 *                     fp8_quant_act_1x128 gives them
 *   FP8BS_CACHE_FP4   as above: e is the smallest with amax <= 6 * 2^e of the
 *                     group, at least -126 (0 for a group of zeros); codes are
 *                     x / 2^e rounded to nearest, halfway to the even code
 * Numbers must be finite. A token whose position is below 0 or past the table,
 * or whose table entry is not in [0, pages), is not written. No two tokens of
 * a call may go to one slot (pages that requests share are only read); what
 * such a slot then holds is not defined. All other slots keep what they hold.
 * Strides: multiples of 8, at least a token's numbers, below 2^31. page >= 1; pages * page
 * below 2^31.
 */
FP8BS_API int fp8bs_mla_cache_write(const uint16_t* latent, int64_t latent_stride, const uint16_t* rope,
                      int64_t rope_stride, const int32_t* cu, int B, int64_t T, int cache_kind,
                      void* cache, void* cache_scales, uint16_t* cache_rope, int64_t pages,
                      int page, const int32_t* table, int64_t table_width, const int32_t* lens,
                      void* stream);

/*
 * The reverse: request b's newest cu[b+1] - cu[b] tokens (all of them where
 * that is lens[b]) as BF16, packed, for the up-projection of
 * fp8bs_mla_prefill's keys and values.
 *   latent [T][512], rope [T][64]  BF16, strides as above
 * FP8: code times scale in FP32, rounded to nearest even; BF16 and FP4 exact.
 * Tokens at positions below 0 or past the table give zeros; table entries are
 * clamped into [0, pages). Rows outside cu[0] .. cu[B]-1 are left as they were.
 */
FP8BS_API int fp8bs_mla_cache_read(int cache_kind, const void* cache, const void* cache_scales,
                      const uint16_t* cache_rope, int64_t pages, int page, const int32_t* table,
                      int64_t table_width, const int32_t* lens, const int32_t* cu, int B,
                      int64_t T, uint16_t* latent, int64_t latent_stride, uint16_t* rope,
                      int64_t rope_stride, void* stream);

/*
 * fp8bs_mla_decode and fp8bs_mla_decode_shared over a 4-bit cache: the same
 * results, arguments and limits, with cache, cache_scales and cache_rope as
 * FP8BS_CACHE_FP4 says. A cached number is an exact BF16 operand; scores and
 * sums are FP32, probabilities are rounded to BF16. workspace: at least
 * fp8bs_mla_decode_fp4_workspace_bytes(B, T, H, table_width, page,
 * prefix_pages) bytes for the current device (prefix_pages: 0 without one).
 */
FP8BS_API int fp8bs_mla_decode_fp4(const uint16_t* q, const uint8_t* cache, const uint8_t* cache_scales,
                      const uint16_t* cache_rope, int64_t pages, int page, const int32_t* table,
                      int64_t table_width, const int32_t* lens, int B, int T, int H, float scale,
                      uint16_t* out, float* lse, void* workspace, void* stream);
FP8BS_API int fp8bs_mla_decode_fp4_shared(const uint16_t* q, const uint8_t* cache,
                      const uint8_t* cache_scales, const uint16_t* cache_rope, int64_t pages,
                      int page, const int32_t* prefix_table, int64_t prefix_pages,
                      const int32_t* prefix_len, const int32_t* table, int64_t table_width,
                      const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
                      float* lse, void* workspace, void* stream);
FP8BS_API int64_t fp8bs_mla_decode_fp4_workspace_bytes(int B, int T, int H, int64_t table_width, int page,
                      int64_t prefix_pages);

/*
 * A whole mixture-of-experts layer for a few tokens:
 *   out_t = bf16( sum_{j < topk} w[t][j] * D_e (silu(G_e x_t) * (U_e x_t)) ),  e = topk_ids[t][j],
 * silu(z) = z / (1 + exp(-z)), over the slots whose id lies in [0, E): others
 * (experts that another GPU holds) add nothing. An expert that a token names
 * twice counts with both weights.
 *   x         [T][K]        BF16
 *   topk_ids  [T][topk]     int32        weights [T][topk] float32
 *   w_up      [E][2F][K]    E4M3 codes: rows 0 .. F-1 are G_e, rows F .. 2F-1 U_e
 *   s_up      [E][2F/128][K/128] float32, one per 128 x 128 block (as
 *             fp8_quant_w_128x128 gives codes and scales, expert by expert)
 *   w_down    [E][K][F]     E4M3 codes D_e       s_down [E][K/128][F/128] float32
 *   out       [T][K]        BF16
 * Unlike the grouped GEMMs it does not quantize activations: x and
 * silu(G x) * (U x) (rounded) are BF16 operands, products and all sums FP32,
 * each 128-wide partial sum scaled as it is added. A chosen expert's weights
 * are read once (twice where more than 32 tokens chose it). Inputs finite; a
 * code 0x7F or 0xFF is a NaN.
 * 0 <= T <= 64, 1 <= topk <= 64, 1 <= E <= 1024; K and F multiples of 128, at
 * least 128 (FP8BS_ERR_TOO_LARGE above 2^16). workspace: at least
 * fp8bs_moe_tokens_workspace_bytes(T, topk, K, F) bytes.
 */
FP8BS_API int fp8bs_moe_tokens(const uint16_t* x, int T, int64_t K, const int32_t* topk_ids,
                      const float* weights, int topk, const uint8_t* w_up, const float* s_up,
                      const uint8_t* w_down, const float* s_down, int E, int64_t F, uint16_t* out,
                      void* workspace, void* stream);
FP8BS_API int64_t fp8bs_moe_tokens_workspace_bytes(int T, int topk, int64_t K, int64_t F);

/*
 * Log probabilities of given tokens: for every row x of logits and y = targets[t],
 *   m = max_i x_i, n = log sum_i exp(x_i - m), logprob = (x_y - m) - n,
 *   entropy = n - sum_i p_i (x_i - m) (p_i = exp(x_i - m - n)),
 *   rank = how many entries come before y when ordered by (larger logit, smaller index),
 *   top_ids, top_logprobs: the first `top` entries in that order, (x_i - m) - n.
 *   logits  [T][V] float32 or BF16 (dtype), `stride` numbers from row to row
 *   targets [T] int32: outside [0, V) (no token): logprob 0, rank -1
 *   logprob, entropy [T] float32   rank [T] int32
 *   norm    [T][2] float32: m and n (their sum is the log of the sum of exp(x_i))
 *   top_ids [T][top] int32, top_logprobs [T][top] float32 (NULL where top is 0)
 * Logits may be of any finite size (masks of the type's lowest value, say).
 * Entries of -inf have no probability. A row of nothing else has m = -inf and
 * n = 0, logprob and top_logprobs -inf and entropy 0. A NaN or +inf in a row
 * gives NaN in its logprob (of a token), entropy and n; its rank and
 * alternatives are then some, within range.
 * T >= 0, 1 <= V <= 2^20, 0 <= top <= min(V, 64), V <= stride < 2^31. logits aligned
 * to its type. workspace: fp8bs_logprobs_workspace_bytes(T, V, top) bytes.
 */
FP8BS_API int fp8bs_logprobs(const void* logits, int dtype, int64_t stride, const int32_t* targets,
                      int64_t T, int64_t V, int top, float* logprob, float* entropy, float* norm,
                      int32_t* rank, int32_t* top_ids, float* top_logprobs, void* workspace,
                      void* stream);
FP8BS_API int64_t fp8bs_logprobs_workspace_bytes(int64_t T, int64_t V, int top);

/*
 * Its gradient: with norm and entropy as fp8bs_logprobs wrote them and
 * d_logprob, d_entropy [T] float32 the gradients of logprob and entropy,
 *   d_logits_i = d_logprob * ([i == y] - p_i) - d_entropy * p_i * (log p_i + entropy)
 * (without the first term where targets[t] is no token), in FP32, rounded once
 * to the type of logits. Entries of -inf: p_i = 0 and p_i log p_i = 0; a row of
 * nothing else gets zeros.
 *   d_logits [T][V], of dtype, contiguous, aligned to its type; not the logits'
 *            own memory, which is read while it is written
 */
FP8BS_API int fp8bs_logprobs_bwd(const void* logits, int dtype, int64_t stride, const int32_t* targets,
                      const float* norm, const float* entropy, const float* d_logprob,
                      const float* d_entropy, int64_t T, int64_t V, void* d_logits, void* stream);

/* FP8BS_SERVE_VERSION of the loaded library. */
FP8BS_API int fp8bs_serve_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_SERVE_H */
