// C ABI of the serving operators: host-side argument validation, then the
// launches on the caller's stream. Declarations and the meaning of every
// argument are in include/fp8bs_serve.h.

#include "attn_host.h"
#include "fp8bs_serve.h"
#include "serve_internal.h"

namespace {

constexpr DecodeShape kShape{fp8bs::kFp4Tile, fp8bs::kFp4BlockRows};

// What the cache's two directions have in common.
int cache_args(int kind, const void* cache, const void* scales, const void* rope_cache, int64_t pages, int page,
               const int32_t* table, int64_t width, const int32_t* lens, const int32_t* cu, int B, int64_t T,
               const uint16_t* latent, int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
               fp8bs::MlaCache& c) {
  if (kind != FP8BS_CACHE_BF16 && kind != FP8BS_CACHE_FP8 && kind != FP8BS_CACHE_FP4) return FP8BS_ERR_MODE;
  if (B < 0 || T < 0 || pages < 0 || page < 1 || width < 0) return FP8BS_ERR_SHAPE;
  if (latent_stride < 512 || rope_stride < 64) return FP8BS_ERR_SHAPE;
  if (latent_stride % 8 || rope_stride % 8) return FP8BS_ERR_ALIGN;
  if (pages > (kI32 - 1) / page || width > (kI32 - 1) / page || T >= kI32 - 64 || B >= 1 << 30)
    return FP8BS_ERR_TOO_LARGE;
  if (launch_too_large((T + 3) / 4, 256)) return FP8BS_ERR_TOO_LARGE;
  if (latent_stride >= kI32 || rope_stride >= kI32) return FP8BS_ERR_TOO_LARGE;
  if (B == 0 || T == 0) return FP8BS_OK;
  if (!latent || !rope || !cu || !lens) return FP8BS_ERR_NULL_PTR;
  if (width > 0 && !table) return FP8BS_ERR_NULL_PTR;
  if (width > 0 && pages == 0) return FP8BS_ERR_SHAPE;       // a table into no pages
  if (width > 0 && (!cache || (kind != FP8BS_CACHE_BF16 && (!scales || !rope_cache)))) return FP8BS_ERR_NULL_PTR;
  if (off16(latent) || off16(rope) || off16(cache)) return FP8BS_ERR_ALIGN;
  if (kind != FP8BS_CACHE_BF16 && (off16(scales) || off16(rope_cache))) return FP8BS_ERR_ALIGN;
  if (off4(cu) || off4(table) || off4(lens)) return FP8BS_ERR_ALIGN;
  c.kind = kind;
  c.cache = static_cast<char*>(const_cast<void*>(cache));
  c.scales = static_cast<char*>(const_cast<void*>(scales));
  c.rope = static_cast<char*>(const_cast<void*>(rope_cache));
  c.latent = const_cast<uint16_t*>(latent);
  c.out_rope = const_cast<uint16_t*>(rope);
  c.latent_stride = latent_stride;
  c.rope_stride = rope_stride;
  c.cu = cu;
  c.table = table;
  c.lens = lens;
  c.width = width;
  c.B = B;
  c.T = (int)T;
  c.pages = (int)pages;
  c.page = page;
  c.max_len = width * page;
  const PageDiv div(page);
  c.page_magic = div.magic;
  c.page_shift = div.shift;
  return FP8BS_OK;
}

int decode4(const uint16_t* q, const uint8_t* cache, const uint8_t* scales, const uint16_t* rope, int64_t pages,
            int page, const int32_t* prefix_table, int64_t prefix_pages, const int32_t* prefix_len,
            const int32_t* table, int64_t width, const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
            float* lse, void* workspace, void* stream) {
  DecodeSizes own{}, prefix{};
  const int st = decode_plan(kShape, B, T, H, width, page, prefix_pages, own, prefix);
  if (st != FP8BS_OK) return st;
  if (pages < 0) return FP8BS_ERR_SHAPE;
  if (pages > (kI32 - 1) / page) return FP8BS_ERR_TOO_LARGE;
  if (bad_scale(scale)) return FP8BS_ERR_VALUE;
  if (B == 0) return FP8BS_OK;
  const bool reads = width > 0 || prefix_pages > 0;
  if (reads && pages == 0) return FP8BS_ERR_SHAPE;       // a table into no pages
  if (!q || !lens || !out || !lse || !workspace) return FP8BS_ERR_NULL_PTR;
  if (width > 0 && !table) return FP8BS_ERR_NULL_PTR;
  if (prefix_pages > 0 && (!prefix_table || !prefix_len)) return FP8BS_ERR_NULL_PTR;
  if (reads && (!cache || !scales || !rope)) return FP8BS_ERR_NULL_PTR;
  if (off16(q) || off16(cache) || off16(scales) || off16(rope) || off16(out) || off16(workspace)) return FP8BS_ERR_ALIGN;
  if (off4(table) || off4(lens) || off4(lse) || off4(prefix_table) || off4(prefix_len)) return FP8BS_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  fp8bs::MlaDecode a{}, b{};
  const bool join = prefix_pages > 0;
  fill(a, q, cache, scales, rope, pages, page, table, width, lens, own, scale, out, lse, join, ws);
  a.tokens = T;
  a.heads = H;
  if (join) {
    fill(b, q, cache, scales, rope, pages, page, prefix_table, 0, prefix_len, prefix, scale, out, lse, true, ws);
    b.len_stride = 0;
    b.tokens = 1;              // it hides nothing
    b.heads = b.rows;
  }
  return status_of(fp8bs::launch_mla_decode_fp4(a, join ? &b : nullptr, as_stream(stream)));
}

int logprobs_sizes(int64_t T, int64_t V, int top) {
  if (T < 0 || V < 1 || top < 0 || top > V || top > 64) return FP8BS_ERR_SHAPE;
  if (V > 1 << 20) return FP8BS_ERR_TOO_LARGE;
  if (T >= kI32 || launch_too_large(T * fp8bs::logprobs_chunks(V), fp8bs::kLogprobsThreads)) return FP8BS_ERR_TOO_LARGE;
  return FP8BS_OK;
}

// Aligned to a number of the type.
bool off_type(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == FP8BS_BF16 ? 1u : 3u)) != 0; }

}  // namespace

extern "C" {

int fp8bs_serve_version(void) { return FP8BS_SERVE_VERSION; }

int fp8bs_mla_cache_write(const uint16_t* latent, int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
                          const int32_t* cu, int B, int64_t T, int cache_kind, void* cache, void* cache_scales,
                          uint16_t* cache_rope, int64_t pages, int page, const int32_t* table, int64_t table_width,
                          const int32_t* lens, void* stream) {
  fp8bs::MlaCache c{};
  const int st = cache_args(cache_kind, cache, cache_scales, cache_rope, pages, page, table, table_width, lens, cu, B,
                            T, latent, latent_stride, rope, rope_stride, c);
  if (st != FP8BS_OK || B == 0 || T == 0 || table_width == 0) return st;
  return status_of(fp8bs::launch_mla_cache_write(c, as_stream(stream)));
}

int fp8bs_mla_cache_read(int cache_kind, const void* cache, const void* cache_scales, const uint16_t* cache_rope,
                         int64_t pages, int page, const int32_t* table, int64_t table_width, const int32_t* lens,
                         const int32_t* cu, int B, int64_t T, uint16_t* latent, int64_t latent_stride, uint16_t* rope,
                         int64_t rope_stride, void* stream) {
  fp8bs::MlaCache c{};
  const int st = cache_args(cache_kind, cache, cache_scales, cache_rope, pages, page, table, table_width, lens, cu, B,
                            T, latent, latent_stride, rope, rope_stride, c);
  if (st != FP8BS_OK || B == 0 || T == 0) return st;
  return status_of(fp8bs::launch_mla_cache_read(c, as_stream(stream)));
}

int64_t fp8bs_mla_decode_fp4_workspace_bytes(int B, int T, int H, int64_t table_width, int page, int64_t prefix_pages) {
  DecodeSizes own{}, prefix{};
  const int st = decode_plan(kShape, B, T, H, table_width, page, prefix_pages, own, prefix);
  if (st != FP8BS_OK) return st;
  return own.bytes() + (prefix_pages > 0 ? prefix.bytes() : 0);
}

int fp8bs_mla_decode_fp4(const uint16_t* q, const uint8_t* cache, const uint8_t* cache_scales,
                         const uint16_t* cache_rope, int64_t pages, int page, const int32_t* table,
                         int64_t table_width, const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
                         float* lse, void* workspace, void* stream) {
  return decode4(q, cache, cache_scales, cache_rope, pages, page, nullptr, 0, nullptr, table, table_width, lens, B, T,
                 H, scale, out, lse, workspace, stream);
}

int fp8bs_mla_decode_fp4_shared(const uint16_t* q, const uint8_t* cache, const uint8_t* cache_scales,
                                const uint16_t* cache_rope, int64_t pages, int page, const int32_t* prefix_table,
                                int64_t prefix_pages, const int32_t* prefix_len, const int32_t* table,
                                int64_t table_width, const int32_t* lens, int B, int T, int H, float scale,
                                uint16_t* out, float* lse, void* workspace, void* stream) {
  return decode4(q, cache, cache_scales, cache_rope, pages, page, prefix_table, prefix_pages, prefix_len, table,
                 table_width, lens, B, T, H, scale, out, lse, workspace, stream);
}

int64_t fp8bs_moe_tokens_workspace_bytes(int T, int topk, int64_t K, int64_t F) {
  if (T < 0 || T > fp8bs::kMoeMaxTokens || topk < 1 || topk > fp8bs::kMoeMaxTopk || K < 128 || K % 128 || F < 128 || F % 128)
    return FP8BS_ERR_SHAPE;
  if (K > 1 << 16 || F > 1 << 16) return FP8BS_ERR_TOO_LARGE;
  return align256((int64_t)2 * T * topk * F) + 4 * fp8bs::moe_shares(K) * T * K;
}

int fp8bs_moe_tokens(const uint16_t* x, int T, int64_t K, const int32_t* topk_ids, const float* weights, int topk,
                     const uint8_t* w_up, const float* s_up, const uint8_t* w_down, const float* s_down, int E,
                     int64_t F, uint16_t* out, void* workspace, void* stream) {
  const int64_t bytes = fp8bs_moe_tokens_workspace_bytes(T, topk, K, F);
  if (bytes < 0) return (int)bytes;
  if (E < 1 || E > fp8bs::kMoeMaxExperts) return FP8BS_ERR_SHAPE;
  if (T == 0) return FP8BS_OK;
  if (!x || !topk_ids || !weights || !w_up || !s_up || !w_down || !s_down || !out || !workspace)
    return FP8BS_ERR_NULL_PTR;
  if (off16(x) || off16(w_up) || off16(w_down) || off16(out) || off16(workspace)) return FP8BS_ERR_ALIGN;
  if (off4(topk_ids) || off4(weights) || off4(s_up) || off4(s_down)) return FP8BS_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  fp8bs::MoeTokens m{};
  m.x = x;
  m.ids = topk_ids;
  m.weights = weights;
  m.w_up = w_up;
  m.s_up = s_up;
  m.w_down = w_down;
  m.s_down = s_down;
  m.h = reinterpret_cast<uint16_t*>(ws);
  m.part = reinterpret_cast<float*>(ws + align256((int64_t)2 * T * topk * F));
  m.out = out;
  m.T = T;
  m.topk = topk;
  m.E = E;
  m.K = (int)K;
  m.F = (int)F;
  m.shares = fp8bs::moe_shares(K);
  return status_of(fp8bs::launch_moe_tokens(m, as_stream(stream)));
}

int64_t fp8bs_logprobs_workspace_bytes(int64_t T, int64_t V, int top) {
  const int st = logprobs_sizes(T, V, top);
  if (st != FP8BS_OK) return st;
  const int64_t chunks = fp8bs::logprobs_chunks(V);
  return T * chunks * (16 + 8 * (int64_t)top);
}

int fp8bs_logprobs(const void* logits, int dtype, int64_t stride, const int32_t* targets, int64_t T, int64_t V,
                   int top, float* logprob, float* entropy, float* norm, int32_t* rank, int32_t* top_ids,
                   float* top_logprobs, void* workspace, void* stream) {
  if (dtype != FP8BS_F32 && dtype != FP8BS_BF16) return FP8BS_ERR_DTYPE;
  const int st = logprobs_sizes(T, V, top);
  if (st != FP8BS_OK) return st;
  if (stride < V) return FP8BS_ERR_SHAPE;
  if (stride >= kI32) return FP8BS_ERR_TOO_LARGE;
  if (T == 0) return FP8BS_OK;
  if (!logits || !targets || !logprob || !entropy || !norm || !rank || !workspace) return FP8BS_ERR_NULL_PTR;
  if (top > 0 && (!top_ids || !top_logprobs)) return FP8BS_ERR_NULL_PTR;
  if (off_type(logits, dtype) || off4(targets) || off4(logprob) || off4(entropy) || off4(norm) || off4(rank) ||
      off4(top_ids) || off4(top_logprobs) || off16(workspace))
    return FP8BS_ERR_ALIGN;
  fp8bs::Logprobs l{};
  l.logits = logits;
  l.stride = stride;
  l.targets = targets;
  l.T = T;
  l.V = (int)V;
  l.top = top;
  l.logprob = logprob;
  l.entropy = entropy;
  l.norm = norm;
  l.rank = rank;
  l.top_ids = top_ids;
  l.top_logprobs = top_logprobs;
  l.part = static_cast<float4*>(workspace);
  l.part_top = reinterpret_cast<uint64_t*>(l.part + T * fp8bs::logprobs_chunks(V));
  return status_of(fp8bs::launch_logprobs(l, dtype == FP8BS_BF16, as_stream(stream)));
}

int fp8bs_logprobs_bwd(const void* logits, int dtype, int64_t stride, const int32_t* targets, const float* norm,
                       const float* entropy, const float* d_logprob, const float* d_entropy, int64_t T, int64_t V,
                       void* d_logits, void* stream) {
  if (dtype != FP8BS_F32 && dtype != FP8BS_BF16) return FP8BS_ERR_DTYPE;
  const int st = logprobs_sizes(T, V, 0);
  if (st != FP8BS_OK) return st;
  if (stride < V) return FP8BS_ERR_SHAPE;
  if (stride >= kI32) return FP8BS_ERR_TOO_LARGE;
  if (T == 0) return FP8BS_OK;
  if (!logits || !targets || !norm || !entropy || !d_logprob || !d_entropy || !d_logits) return FP8BS_ERR_NULL_PTR;
  if (off_type(logits, dtype) || off_type(d_logits, dtype) || off4(targets) || off4(norm) || off4(entropy) ||
      off4(d_logprob) || off4(d_entropy))
    return FP8BS_ERR_ALIGN;
  fp8bs::Logprobs l{};
  l.logits = logits;
  l.stride = stride;
  l.targets = targets;
  l.T = T;
  l.V = (int)V;
  l.norm = const_cast<float*>(norm);
  l.entropy = const_cast<float*>(entropy);
  l.d_logprob = d_logprob;
  l.d_entropy = d_entropy;
  l.d_logits = d_logits;
  return status_of(fp8bs::launch_logprobs_bwd(l, dtype == FP8BS_BF16, as_stream(stream)));
}

}  // extern "C"
