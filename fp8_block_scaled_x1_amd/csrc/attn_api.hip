// C ABI of the attention and draft-verification operators: host-side argument
// validation, then the launches on the caller's stream. Declarations and the
// meaning of every argument are in include/fp8bs_attn.h.

#include "attn_host.h"

namespace {

constexpr DecodeShape kShape{fp8bs::kMlaDecodeTile, fp8bs::kMlaDecodeBlockRows};

int prefill_sizes(int B, int64_t Tq, int64_t Tk, int H, int64_t q_stride, int64_t kv_stride, int64_t rope_stride,
                  float scale) {
  if (B < 0 || Tq < 0 || Tk < 0 || H < 1) return FP8BS_ERR_SHAPE;
  if (B == 0 && (Tq > 0 || Tk > 0)) return FP8BS_ERR_SHAPE;      // tokens of no request
  if (H > 32768 || Tq >= kI32 - 65536 || Tk >= kI32 - 65536) return FP8BS_ERR_TOO_LARGE;
  if (q_stride < (int64_t)H * 192 || kv_stride < (int64_t)H * 256 || rope_stride < 64) return FP8BS_ERR_SHAPE;
  if (q_stride % 8 || kv_stride % 8 || rope_stride % 8) return FP8BS_ERR_ALIGN;
  // a tile's rows are addressed by 32-bit byte offsets from its first
  if (q_stride >= 1 << 24 || kv_stride >= 1 << 24 || rope_stride >= 1 << 24) return FP8BS_ERR_TOO_LARGE;
  // (the forward's narrower blocks have half the threads and are at most twice as many)
  if (launch_too_large(fp8bs::mla_blocks(Tq, B, 256) * H, 512)) return FP8BS_ERR_TOO_LARGE;
  if (bad_scale(scale)) return FP8BS_ERR_VALUE;
  return FP8BS_OK;
}

int decode(const uint16_t* q, int kind, const void* cache, const float* scales, const uint16_t* rope, int64_t pages,
           int page, const int32_t* prefix_table, int64_t prefix_pages, const int32_t* prefix_len,
           const int32_t* table, int64_t width, const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
           float* lse, void* workspace, void* stream) {
  if (kind != FP8BS_CACHE_BF16 && kind != FP8BS_CACHE_FP8) return FP8BS_ERR_MODE;
  DecodeSizes own{}, prefix{};
  const int st = decode_plan(kShape, B, T, H, width, page, prefix_pages, own, prefix);
  if (st != FP8BS_OK) return st;
  if (pages < 0) return FP8BS_ERR_SHAPE;
  if (pages >= kI32) return FP8BS_ERR_TOO_LARGE;
  if (bad_scale(scale)) return FP8BS_ERR_VALUE;
  if (B == 0) return FP8BS_OK;
  const bool reads = width > 0 || prefix_pages > 0;
  if (reads && pages == 0) return FP8BS_ERR_SHAPE;       // a table into no pages
  if (!q || !lens || !out || !lse || !workspace) return FP8BS_ERR_NULL_PTR;
  if (width > 0 && !table) return FP8BS_ERR_NULL_PTR;
  if (prefix_pages > 0 && (!prefix_table || !prefix_len)) return FP8BS_ERR_NULL_PTR;
  if (reads && (!cache || (kind == FP8BS_CACHE_FP8 && (!scales || !rope)))) return FP8BS_ERR_NULL_PTR;
  if (off16(q) || off16(cache) || off16(out) || off16(workspace)) return FP8BS_ERR_ALIGN;
  if (kind == FP8BS_CACHE_FP8 && (off16(scales) || off16(rope))) return FP8BS_ERR_ALIGN;
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
  return status_of(fp8bs::launch_mla_decode(a, join ? &b : nullptr, kind == FP8BS_CACHE_FP8, as_stream(stream)));
}

}  // namespace

extern "C" {

int fp8bs_attn_version(void) { return FP8BS_ATTN_VERSION; }

int fp8bs_mla_prefill(const uint16_t* q, int64_t q_stride, const uint16_t* kv, int64_t kv_stride,
                      const uint16_t* k_rope, int64_t rope_stride, const int32_t* cu_q, const int32_t* cu_k, int B,
                      int64_t Tq, int64_t Tk, int H, float scale, int causal, uint16_t* out, float* lse,
                      void* workspace, void* stream) {
  const int st = prefill_sizes(B, Tq, Tk, H, q_stride, kv_stride, rope_stride, scale);
  if (st != FP8BS_OK) return st;
  if (Tq == 0) return FP8BS_OK;
  if (!q || !cu_q || !cu_k || !out || !lse || (Tk > 0 && (!kv || !k_rope))) return FP8BS_ERR_NULL_PTR;
  if (off16(q) || off16(kv) || off16(k_rope) || off16(out)) return FP8BS_ERR_ALIGN;
  if (off4(cu_q) || off4(cu_k) || off4(lse)) return FP8BS_ERR_ALIGN;
  const int parts = fp8bs::mla_prefill_parts(B, Tq, Tk, H);
  if (parts > 1 && !workspace) return FP8BS_ERR_NULL_PTR;
  if (parts > 1 && off16(workspace)) return FP8BS_ERR_ALIGN;
  fp8bs::MlaPrefill p{};
  p.parts = parts;
  p.part = static_cast<float*>(workspace);
  p.part_ml = parts > 1 ? p.part + parts * Tq * H * 128 : nullptr;
  p.q = q; p.kv = kv; p.k_rope = k_rope;
  p.q_stride = q_stride; p.kv_stride = kv_stride; p.rope_stride = rope_stride;
  p.cu_q = cu_q; p.cu_k = cu_k;
  p.B = B; p.H = H; p.Tq = (int)Tq; p.Tk = (int)Tk;
  p.scale = scale;
  p.causal = causal != 0;
  p.out = out;
  p.lse = lse;
  return status_of(fp8bs::launch_mla_prefill(p, as_stream(stream)));
}

int64_t fp8bs_mla_prefill_workspace_bytes(int B, int64_t Tq, int64_t Tk, int H) {
  if (B < 0 || Tq < 0 || Tk < 0 || H < 1) return FP8BS_ERR_SHAPE;
  if (Tq >= kI32 || Tk >= kI32 || H > 32768) return FP8BS_ERR_TOO_LARGE;
  const int parts = fp8bs::mla_prefill_parts(B, Tq, Tk, H);
  return parts > 1 ? parts * Tq * H * (128 + 2) * 4 : 0;
}

int64_t fp8bs_mla_prefill_bwd_workspace_bytes(int64_t Tq, int64_t Tk, int H) {
  if (Tq < 0 || Tk < 0 || H < 1) return FP8BS_ERR_SHAPE;
  if (Tq >= kI32 || Tk >= kI32 || H > 32768) return FP8BS_ERR_TOO_LARGE;
  return 2 * align256(4 * Tq * H) + 4 * Tk * H * 64;
}

int fp8bs_mla_prefill_bwd(const uint16_t* dout, const uint16_t* q, int64_t q_stride, const uint16_t* kv,
                          int64_t kv_stride, const uint16_t* k_rope, int64_t rope_stride, const uint16_t* out,
                          const float* lse, const int32_t* cu_q, const int32_t* cu_k, int B, int64_t Tq, int64_t Tk,
                          int H, float scale, int causal, uint16_t* dq, uint16_t* dkv, uint16_t* dk_rope,
                          void* workspace, void* stream) {
  const int st = prefill_sizes(B, Tq, Tk, H, q_stride, kv_stride, rope_stride, scale);
  if (st != FP8BS_OK) return st;
  if (launch_too_large(fp8bs::mla_blocks(Tq, B, 128) * H, 256) ||
      launch_too_large(fp8bs::mla_blocks(Tk, B, 128) * H, 512) || launch_too_large(Tk, 64))
    return FP8BS_ERR_TOO_LARGE;
  if (Tq == 0 && Tk == 0) return FP8BS_OK;
  if (!cu_q || !cu_k || !workspace) return FP8BS_ERR_NULL_PTR;
  if (Tq > 0 && (!dout || !q || !out || !lse || !dq)) return FP8BS_ERR_NULL_PTR;
  if (Tk > 0 && (!kv || !k_rope || !dkv || !dk_rope)) return FP8BS_ERR_NULL_PTR;
  if (off16(dout) || off16(q) || off16(kv) || off16(k_rope) || off16(out) || off16(dq) || off16(dkv) ||
      off16(dk_rope) || off16(workspace))
    return FP8BS_ERR_ALIGN;
  if (off4(cu_q) || off4(cu_k) || off4(lse)) return FP8BS_ERR_ALIGN;
  fp8bs::MlaPrefill p{};
  p.q = q; p.kv = kv; p.k_rope = k_rope;
  p.q_stride = q_stride; p.kv_stride = kv_stride; p.rope_stride = rope_stride;
  p.cu_q = cu_q; p.cu_k = cu_k;
  p.B = B; p.H = H; p.Tq = (int)Tq; p.Tk = (int)Tk;
  p.scale = scale;
  p.causal = causal != 0;
  p.out = const_cast<uint16_t*>(out);
  p.lse = const_cast<float*>(lse);
  p.dout = dout;
  p.delta = static_cast<float*>(workspace);
  p.lse2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256(4 * Tq * H));
  p.rope_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + 2 * align256(4 * Tq * H));
  p.dq = dq; p.dkv = dkv; p.dk_rope = dk_rope;
  return status_of(fp8bs::launch_mla_prefill_bwd(p, as_stream(stream)));
}

int64_t fp8bs_mla_decode_workspace_bytes(int B, int T, int H, int64_t table_width, int page, int64_t prefix_pages) {
  DecodeSizes own{}, prefix{};
  const int st = decode_plan(kShape, B, T, H, table_width, page, prefix_pages, own, prefix);
  if (st != FP8BS_OK) return st;
  return own.bytes() + (prefix_pages > 0 ? prefix.bytes() : 0);
}

int fp8bs_mla_decode(const uint16_t* q, int cache_kind, const void* cache, const float* cache_scales,
                     const uint16_t* cache_rope, int64_t pages, int page, const int32_t* table, int64_t table_width,
                     const int32_t* lens, int B, int T, int H, float scale, uint16_t* out, float* lse,
                     void* workspace, void* stream) {
  return decode(q, cache_kind, cache, cache_scales, cache_rope, pages, page, nullptr, 0, nullptr, table, table_width,
                lens, B, T, H, scale, out, lse, workspace, stream);
}

int fp8bs_mla_decode_shared(const uint16_t* q, int cache_kind, const void* cache, const float* cache_scales,
                            const uint16_t* cache_rope, int64_t pages, int page, const int32_t* prefix_table,
                            int64_t prefix_pages, const int32_t* prefix_len, const int32_t* table,
                            int64_t table_width, const int32_t* lens, int B, int T, int H, float scale, uint16_t* out,
                            float* lse, void* workspace, void* stream) {
  return decode(q, cache_kind, cache, cache_scales, cache_rope, pages, page, prefix_table, prefix_pages, prefix_len,
                table, table_width, lens, B, T, H, scale, out, lse, workspace, stream);
}

int64_t fp8bs_verify_drafts_workspace_bytes(int B, int64_t V) {
  if (B < 0 || V < 1) return FP8BS_ERR_SHAPE;
  if (V > 1 << 24) return FP8BS_ERR_TOO_LARGE;
  const int64_t chunks = fp8bs::verify_chunks(V);
  if (launch_too_large(B * chunks, fp8bs::kVerifyThreads)) return FP8BS_ERR_TOO_LARGE;
  return (int64_t)16 * B * (chunks + 1);
}

int fp8bs_verify_drafts(const void* p, const void* q, int dtype, const int32_t* drafts, const int32_t* n_drafts,
                        const float* u, const float* u_next, int B, int K, int64_t V, int32_t* tokens,
                        int32_t* accepted, void* workspace, void* stream) {
  if (dtype != FP8BS_F32 && dtype != FP8BS_BF16) return FP8BS_ERR_DTYPE;
  if (K < 0 || K > 63) return FP8BS_ERR_SHAPE;
  const int64_t bytes = fp8bs_verify_drafts_workspace_bytes(B, V);
  if (bytes < 0) return (int)bytes;
  if (B == 0) return FP8BS_OK;
  if (!p || !n_drafts || !u_next || !tokens || !accepted || !workspace) return FP8BS_ERR_NULL_PTR;
  if (K > 0 && (!drafts || !u)) return FP8BS_ERR_NULL_PTR;
  if (off4(p) || off4(q) || off4(drafts) || off4(n_drafts) || off4(u) || off4(u_next) || off4(tokens) ||
      off4(accepted) || off16(workspace))
    return FP8BS_ERR_ALIGN;
  fp8bs::VerifyDrafts v{};
  v.p = p; v.q = q;
  v.drafts = drafts; v.n_drafts = n_drafts;
  v.u = u; v.u_next = u_next;
  v.B = B; v.K = K; v.V = (int)V;
  v.rows = static_cast<int4*>(workspace);
  v.sums = reinterpret_cast<uint64_t*>(v.rows + B);
  v.tokens = tokens; v.accepted = accepted;
  return status_of(fp8bs::launch_verify_drafts(v, dtype == FP8BS_BF16, as_stream(stream)));
}

}  // extern "C"
