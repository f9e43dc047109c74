/*
 * fp8bs_attn.h -- attention and decoding operators of libfp8bs.so (gfx950),
 * next to the FP8 GEMMs of fp8bs.h: latent attention in its expanded form
 * (prefill and training, forward and backward) and in its absorbed form over a
 * paged cache (decoding), the latter also for a batch behind a common prefix,
 * and the verification of drafted tokens.
 *
 * Conventions as in fp8bs.h: device pointers to caller-owned memory, work
 * enqueued on `stream` without synchronizing, arguments checked on the host
 * before anything is enqueued, an fp8bs_status returned. The library allocates
 * nothing; workspaces are the caller's, sized by the *_workspace_bytes
 * functions, their contents on entry do not matter. Every entry point can be
 * captured into a HIP graph and gives the same bits for the same inputs.
 * Sizes whose launch would pass 2^32 - 1 threads are refused (FP8BS_ERR_TOO_LARGE).
 * Pointers are 16-byte aligned unless said otherwise; int32 and float32 side
 * arrays (offsets, lengths, tables, random numbers, lse) 4-byte. Numbers that
 * take part in an attention's result should be finite: a NaN among those that a
 * score is formed from makes out and lse of the queries that see it NaN (they
 * do not pass for queries that see no key). What lies past a request's length,
 * in a page's unused slots or behind unused table entries is never used.
 *
 * Dimensions: a head has 128 + 64 query and key numbers (the 64 rotary ones of
 * the key shared by all heads) and 128 value numbers; the cached latent vector
 * has 512 numbers, with the 64 rotary ones 576.
 */
#ifndef FP8BS_ATTN_H
#define FP8BS_ATTN_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BS_ATTN_VERSION 1

/* A scalar argument is outside its range (in addition to fp8bs_status). */
#define FP8BS_ERR_VALUE (-9)

/* What the paged cache holds (see fp8bs_mla_decode). */
enum fp8bs_cache { FP8BS_CACHE_BF16 = 0, FP8BS_CACHE_FP8 = 1 };

/*
 * Latent attention, expanded form, for B requests packed one after the other:
 * request b has the queries cu_q[b] .. cu_q[b+1]-1 and the keys cu_k[b] ..
 * cu_k[b+1]-1. For every head h, query i and key j of one request (numbered
 * inside it, Lq and Lk of them),
 *   S_ij = scale * (q_i[h][0:128] . kv_j[h][0:128] + q_i[h][128:192] . k_rope_j)
 *   out_i[h] = sum_j softmax_j(S_ij) * kv_j[h][128:256],  lse[h][i] = log sum_j exp(S_ij)
 * over all keys, or with causal != 0 over j <= i + Lk - Lq: the last query sees
 * every key, so Lk > Lq is a chunk behind Lk - Lq cached tokens. A query that
 * sees no key (Lk == 0, or causal with Lk < Lq) gets out = 0 and lse = -inf.
 *   q       [Tq][H][192]  BF16, q_stride numbers from token to token
 *   kv      [Tk][H][256]  BF16, kv_stride numbers from token to token: keys
 *                         (128) then values (128) of each head
 *   k_rope  [Tk][64]      BF16, rope_stride numbers from token to token
 *   cu_q, cu_k [B+1]      int32: first is 0, non-decreasing, last is Tq (Tk)
 *                         (precondition; the kernels clamp them into range)
 *   out     [Tq][H][128]  BF16      lse [H][Tq] float32
 * Strides: multiples of 8, at least a token's numbers, below 2^24. Scores, statistics and
 * sums are FP32; probabilities are rounded to BF16 for the matrix unit.
 * A request's own keys and values are finite: one that a query does not see has
 * weight 0, and 0 * inf is NaN. Other requests' numbers do not matter.
 * scale finite and > 0 (else FP8BS_ERR_VALUE); H >= 1. workspace: at least
 * fp8bs_mla_prefill_workspace_bytes(B, Tq, Tk, H) bytes, for the parts of few
 * queries' many keys (0 bytes where there are none: then it may be NULL).
 */
FP8BS_API int fp8bs_mla_prefill(const uint16_t* q, int64_t q_stride, const uint16_t* kv, int64_t kv_stride,
                      const uint16_t* k_rope, int64_t rope_stride, const int32_t* cu_q,
                      const int32_t* cu_k, int B, int64_t Tq, int64_t Tk, int H, float scale,
                      int causal, uint16_t* out, float* lse, void* workspace, void* stream);
FP8BS_API int64_t fp8bs_mla_prefill_workspace_bytes(int B, int64_t Tq, int64_t Tk, int H);

/*
 * Its gradients: with out and lse as fp8bs_mla_prefill wrote them for the same
 * arguments and dout the gradient of out,
 *   dq     [Tq][H][192], dkv [Tk][H][256], dk_rope [Tk][64] (summed over the
 *          heads in FP32)    BF16, contiguous
 * Keys that no query sees get zeros, and so do queries that see no key.
 * dout [Tq][H][128] contiguous. workspace: at least
 * fp8bs_mla_prefill_bwd_workspace_bytes(Tq, Tk, H) bytes.
 */
FP8BS_API int fp8bs_mla_prefill_bwd(const uint16_t* dout, const uint16_t* q, int64_t q_stride,
                      const uint16_t* kv, int64_t kv_stride, const uint16_t* k_rope,
                      int64_t rope_stride, const uint16_t* out, const float* lse,
                      const int32_t* cu_q, const int32_t* cu_k, int B, int64_t Tq, int64_t Tk,
                      int H, float scale, int causal, uint16_t* dq, uint16_t* dkv,
                      uint16_t* dk_rope, void* workspace, void* stream);
FP8BS_API int64_t fp8bs_mla_prefill_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int H);

/*
 * Latent attention, absorbed form: T query tokens of each of B requests (their
 * newest; T > 1 scores drafted tokens) against the request's cached vectors
 * c_j = (latent 512 | rotary 64), which every head shares and whose latent
 * part is also the value:
 *   S_j = scale * q[b][t][h] . c_j,  out[b][t][h] = sum_j softmax_j(S_j) * c_j[0:512]
 * over j < lens[b] - (T - 1 - t). A query that sees no token gets out = 0 and
 * lse = -inf.
 *   q      [B][T][H][576] BF16     out [B][T][H][512] BF16    lse [B][T][H] float32
 *   cache  FP8BS_CACHE_BF16: BF16 [pages][page][576]; cache_scales and
 *          cache_rope unused (NULL)
 *          FP8BS_CACHE_FP8: E4M3 codes [pages][page][512] of the latent
 *          numbers, their scales cache_scales float32 [pages][page][4], one per
 *          128 (codes and scales as fp8_quant_act_1x128 gives them, the scales
 *          transposed: here a token's four lie together),
 *          and cache_rope BF16 [pages][page][64]
 *   table  [B][table_width] int32: token j of request b is in slot j % page of
 *          page table[b][j / page]; entries are clamped into [0, pages), those
 *          past a request's last token are not read
 *   lens   [B] int32, clamped into [0, table_width * page]
 * page >= 1, any; T, H >= 1. workspace: at least
 * fp8bs_mla_decode_workspace_bytes(B, T, H, table_width, page, 0) bytes for
 * the current device.
 */
FP8BS_API int fp8bs_mla_decode(const uint16_t* q, int cache_kind, const void* cache,
                      const float* cache_scales, const uint16_t* cache_rope, int64_t pages,
                      int page, const int32_t* table, int64_t table_width, const int32_t* lens,
                      int B, int T, int H, float scale, uint16_t* out, float* lse,
                      void* workspace, void* stream);

/*
 * The same for requests that all begin with one common prefix, whose
 * prefix_len[0] tokens lie in the pages prefix_table[0 .. prefix_pages-1] of
 * the same cache (prefix_len: DEVICE int32[1], clamped into [0, prefix_pages *
 * page]); table and lens hold each request's own tokens after it (at least T
 * of them where every query token is one of them: the prefix hides nothing).
 * The prefix is read once for all requests. Results as if each request's
 * tokens were the prefix and then its own. workspace: sized with the same
 * prefix_pages.
 */
FP8BS_API int fp8bs_mla_decode_shared(const uint16_t* q, int cache_kind, const void* cache,
                      const float* cache_scales, const uint16_t* cache_rope, int64_t pages,
                      int page, const int32_t* prefix_table, int64_t prefix_pages,
                      const int32_t* prefix_len, const int32_t* table, int64_t table_width,
                      const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
                      float* lse, void* workspace, void* stream);
/* Negative: invalid sizes. prefix_pages: 0 for fp8bs_mla_decode. */
FP8BS_API int64_t fp8bs_mla_decode_workspace_bytes(int B, int T, int H, int64_t table_width, int page,
                      int64_t prefix_pages);

/*
 * Verification of drafted tokens. Request b proposed n_drafts[b] <= K tokens
 * drafts[b][j]; draft j is accepted iff u[b][j] * q_j(x) < p_j(x), x the draft,
 * p the target's and q the draft model's probabilities at its position; a
 * draft outside [0, V) is not accepted. The drafts before the first that is
 * not accepted stand (accepted[b] = a of them). The next token is drawn with
 * u_next[b] from max(p_a - q_a, 0) after a rejection (from p_a where that has
 * no weight), from p_a after the last draft:
 *   w_i = floor(min(r_i, 1) * 2^38) (0 where r_i is not positive), W = sum w_i,
 *   token = the first i with w_0 + .. + w_i > floor(W * floor(u_next * 2^24) / 2^24)
 * in whole numbers; -1 if no entry has weight.
 *   p   [B][K+1][V], q [B][K][V]  float32 or BF16 (dtype, both); q NULL: the
 *       drafts were chosen without chance (q_j is 1 at the draft, 0 elsewhere)
 *   drafts [B][K] int32, n_drafts [B] int32 (clamped into [0, K])
 *   u [B][K], u_next [B] float32 in [0, 1)
 *   tokens [B][K+1] int32: the accepted drafts, the next token, then -1
 *   accepted [B] int32
 * 0 <= K <= 63, 1 <= V <= 2^24, B * ceil(V / 8192) < 2^24. p and q 4-byte aligned. workspace:
 * fp8bs_verify_drafts_workspace_bytes(B, V) bytes.
 */
FP8BS_API int fp8bs_verify_drafts(const void* p, const void* q, int dtype, const int32_t* drafts,
                      const int32_t* n_drafts, const float* u, const float* u_next, int B, int K,
                      int64_t V, int32_t* tokens, int32_t* accepted, void* workspace,
                      void* stream);
FP8BS_API int64_t fp8bs_verify_drafts_workspace_bytes(int B, int64_t V);

/* FP8BS_ATTN_VERSION of the loaded library. */
FP8BS_API int fp8bs_attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_ATTN_H */
