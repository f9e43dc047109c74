"""ctypes binding of the serving operators (include/fp8bs_serve.h): argument
marshalling only, as in _attn.

Every function has the name of the C entry point it calls, checks the tensors
it is given, allocates the outputs and the workspace with torch and calls the
library on the current torch stream of the inputs' device. Results carry no
autograd graph: fp8bs_logprobs_bwd gives the gradient of fp8bs_logprobs
(examples/serving_step.py wraps the two in an autograd function).

A paged cache is a tensor BF16 [pages][page][576], or a triple: FP8 (codes uint8
[..][512], scales f32 [..][4], rope bf16 [..][64]) or FP4 (codes uint8
[..][256], scales uint8 [..][16], rope bf16 [..][64]).
"""

import functools

import torch

from . import _attn, _lib
from ._attn import _bf16, _bytes, _bytes_on, _call, _f, _f32, _i, _i32, _i64, _on_gpu, _ptr, _tokens, _u8, _vp, _workspace

SERVE_VERSION = 1
CACHE_FP4 = 2

_SIGNATURES = {
    "fp8bs_mla_cache_write": [_vp, _i64, _vp, _i64, _vp, _i, _i64, _i, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _vp],
    "fp8bs_mla_cache_read": [_i, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _vp, _i, _i64, _vp, _i64, _vp, _i64, _vp],
    "fp8bs_mla_decode_fp4": [_vp, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _i, _i, _i, _f, _vp, _vp, _vp, _vp],
    "fp8bs_mla_decode_fp4_shared": [_vp, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _vp, _i64, _vp, _i, _i, _i, _f, _vp,
                                    _vp, _vp, _vp],
    "fp8bs_mla_decode_fp4_workspace_bytes": [_i, _i, _i, _i64, _i, _i64],
    "fp8bs_moe_tokens": [_vp, _i, _i64, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i64, _vp, _vp, _vp],
    "fp8bs_moe_tokens_workspace_bytes": [_i, _i, _i64, _i64],
    "fp8bs_logprobs": [_vp, _i, _i64, _vp, _i64, _i64, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "fp8bs_logprobs_workspace_bytes": [_i64, _i64, _i],
    "fp8bs_logprobs_bwd": [_vp, _i, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp],
    "fp8bs_serve_version": [],
}

_serve = None

# where sizes alone give the answer
_known_bytes = functools.lru_cache(maxsize=4096)(_bytes)


def serve_lib():
    """The loaded library with the signatures of fp8bs_serve.h."""
    global _serve
    if _serve is None:
        handle = _attn.attn_lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = _i64 if name.endswith("_bytes") else _i
        if handle.fp8bs_serve_version() != SERVE_VERSION:
            raise ImportError(f"libfp8bs serving version {handle.fp8bs_serve_version()} != {SERVE_VERSION}")
        _serve = handle
    return _serve


def _fp4_args(cache, device):
    """(pointers, pages, page size) of an FP4 cache."""
    if not isinstance(cache, (tuple, list)) or len(cache) != 3:
        raise ValueError("an FP4 cache is (codes, scales, rope)")
    codes, scales, rope = cache
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
        raise ValueError("cache codes must be [pages][page][256]")
    n, page = codes.shape[:2]
    return (_ptr(codes, "cache codes", _u8, (n, page, 256), device), _ptr(scales, "cache scales", _u8, (n, page, 16), device),
            _ptr(rope, "cache rope", _bf16, (n, page, 64), device), n, page)


def _any_cache(cache, device):
    """(kind, pointers, pages, page size) of a cache of any kind."""
    if isinstance(cache, (tuple, list)) and len(cache) == 3 and isinstance(cache[0], torch.Tensor) and \
            cache[0].dim() == 3 and cache[0].shape[-1] == 256:
        return (CACHE_FP4, *_fp4_args(cache, device))
    return _attn._cache_args(cache, device)


def _paged(table, lens, cu, device):
    """(table, width, lens, cu, B) of requests with pages and packed rows."""
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("cu must have B+1 entries")
    B = cu.shape[0] - 1
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be [B][width]")
    width = table.shape[1]
    return (_ptr(table, "table", _i32, (B, width), device), width, _ptr(lens, "lens", _i32, (B,), device),
            _ptr(cu, "cu", _i32, (B + 1,), device), B)


def fp8bs_mla_cache_write(latent, rope, cache, table, lens, cu):
    """Puts the requests' newest tokens into their pages, in place: latent BF16
    [T][512] and rope [T][64] (possibly with gaps between tokens) hold request
    b's in the rows cu[b] .. cu[b+1]-1, its positions end at lens[b]. cache: of
    any kind; table int32 [B][width], lens int32 [B], cu int32 [B+1]."""
    serve_lib()
    device = _on_gpu(latent, "latent", (None, 512))
    pl, sl = _tokens(latent, "latent", (512,), device)
    pr, sr = _tokens(rope, "rope", (64,), device)
    if rope.shape[0] != latent.shape[0]:
        raise ValueError("latent and rope disagree on the number of tokens")
    kind, *c = _any_cache(cache, device)
    pt, width, pn, pc, B = _paged(table, lens, cu, device)
    _call("fp8bs_mla_cache_write", device, pl, sl, pr, sr, pc, B, latent.shape[0], kind, *c, pt, width, pn)


def fp8bs_mla_cache_read(cache, table, lens, cu, tokens, out=None):
    """The requests' newest cu[b+1] - cu[b] tokens as BF16, packed: (latent
    [tokens][512], rope [tokens][64]), `tokens` the rows to provide (cu[B] or
    more). out: the two tensors to write to instead of new ones; rows that
    belong to no request are left as they are."""
    serve_lib()
    first = cache[0] if isinstance(cache, (tuple, list)) and cache else cache
    device = _on_gpu(first, "cache", (None, None, None))
    kind, *c = _any_cache(cache, device)
    pt, width, pn, pc, B = _paged(table, lens, cu, device)
    if out is None:
        out = (torch.empty((tokens, 512), dtype=_bf16, device=device), torch.empty((tokens, 64), dtype=_bf16, device=device))
    latent, rope = out
    pl, sl = _tokens(latent, "latent", (512,), device)
    pr, sr = _tokens(rope, "rope", (64,), device)
    if latent.shape[0] != tokens or rope.shape[0] != tokens:
        raise ValueError("out must have `tokens` rows")
    _call("fp8bs_mla_cache_read", device, kind, *c, pt, width, pn, pc, B, tokens, pl, sl, pr, sr)
    return latent, rope


def _decode(fn, q, cache, prefix, table, lens, scale):
    serve_lib()
    device = _on_gpu(q, "q", (None, None, None, 576))
    B, T, H, _ = q.shape
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be [B][width]")
    width = table.shape[1]
    pq = _ptr(q, "q", _bf16, q.shape, device)
    cache_args = _fp4_args(cache, device)
    pre, n_pre = (), 0
    if prefix is not None:
        prefix_table, prefix_len = prefix
        if not isinstance(prefix_table, torch.Tensor) or prefix_table.dim() != 1:
            raise ValueError("prefix_table must be [pages of the prefix]")
        n_pre = prefix_table.shape[0]
        pre = (_ptr(prefix_table, "prefix_table", _i32, (n_pre,), device), n_pre,
               _ptr(prefix_len, "prefix_len", _i32, (1,), device))
    pt, pl = _ptr(table, "table", _i32, (B, width), device), _ptr(lens, "lens", _i32, (B,), device)
    out = torch.empty((B, T, H, 512), dtype=_bf16, device=device)
    lse = torch.empty((B, T, H), dtype=_f32, device=device)
    ws = _workspace(_bytes_on(device.index, "fp8bs_mla_decode_fp4_workspace_bytes", B, T, H, width, cache_args[4], n_pre),
                    device)
    _call(fn, device, pq, *cache_args, *pre, pt, width, pl, B, T, H, float(scale), out.data_ptr(), lse.data_ptr(),
          ws.data_ptr())
    return out, lse


def fp8bs_mla_decode_fp4(q, cache, table, lens, scale):
    """fp8bs_mla_decode over an FP4 cache (codes uint8 [pages][page][256], scales
    uint8 [pages][page][16], rope bf16 [pages][page][64]): q [B][T][H][576] BF16,
    table int32 [B][width], lens int32 [B]. Returns (out bf16 [B][T][H][512], lse
    f32 [B][T][H])."""
    return _decode("fp8bs_mla_decode_fp4", q, cache, None, table, lens, scale)


def fp8bs_mla_decode_fp4_shared(q, cache, prefix_table, prefix_len, table, lens, scale):
    """fp8bs_mla_decode_fp4 for requests that share a prefix of prefix_len[0]
    tokens in the pages prefix_table; table and lens hold each request's own."""
    return _decode("fp8bs_mla_decode_fp4_shared", q, cache, (prefix_table, prefix_len), table, lens, scale)


def fp8bs_moe_tokens(x, topk_ids, weights, w_up, s_up, w_down, s_down):
    """A mixture-of-experts layer for up to 64 tokens: x BF16 [T][K], topk_ids
    int32 [T][topk] (ids outside [0, E) add nothing), weights f32 [T][topk],
    w_up uint8 [E][2F][K] (gate rows, then up rows) and w_down uint8 [E][K][F]
    E4M3 codes with scales f32 [E][2F/128][K/128] and [E][K/128][F/128].
    Returns bf16 [T][K]."""
    serve_lib()
    device = _on_gpu(x, "x", (None, None))
    T, K = x.shape
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [T][topk]")
    if not isinstance(w_down, torch.Tensor) or w_down.dim() != 3 or w_down.shape[1] != K:
        raise ValueError("w_down must be [E][K][F]")
    topk, (E, _, F) = topk_ids.shape[1], w_down.shape
    if K % 128 or F % 128:
        raise ValueError("K and F must be multiples of 128")
    args = (_ptr(x, "x", _bf16, (T, K), device), T, K, _ptr(topk_ids, "topk_ids", _i32, (T, topk), device),
            _ptr(weights, "weights", _f32, (T, topk), device), topk, _ptr(w_up, "w_up", _u8, (E, 2 * F, K), device),
            _ptr(s_up, "s_up", _f32, (E, F // 64, K // 128), device), _ptr(w_down, "w_down", _u8, (E, K, F), device),
            _ptr(s_down, "s_down", _f32, (E, K // 128, F // 128), device), E, F)
    out = torch.empty((T, K), dtype=_bf16, device=device)
    ws = _workspace(_known_bytes("fp8bs_moe_tokens_workspace_bytes", T, topk, K, F), device)
    _call("fp8bs_moe_tokens", device, *args, out.data_ptr(), ws.data_ptr())
    return out


def _rows(logits, targets):
    """(device, dtype code, stride, T, V, pointers) of logits whose rows may lie apart."""
    serve_lib()
    device = _on_gpu(logits, "logits", (None, None))
    T, V = logits.shape
    if logits.dtype not in (_f32, _bf16):
        raise TypeError(f"logits has dtype {logits.dtype}, expected float32 or bfloat16")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the logits of a row must be contiguous")
    stride = logits.stride(0) if T > 1 else V
    if stride < V:
        raise ValueError("rows of logits must not overlap")
    return (device, _lib.BF16 if logits.dtype == _bf16 else _lib.F32, stride, T, V, logits.data_ptr(),
            _ptr(targets, "targets", _i32, (T,), device))


def fp8bs_logprobs(logits, targets, top=0):
    """Log probabilities of given tokens: logits f32 or bf16 [T][V] (rows may lie
    apart), targets int32 [T]. Returns (logprob f32 [T], entropy f32 [T], norm f32
    [T][2], rank int32 [T], top_ids int32 [T][top], top_logprobs f32 [T][top])."""
    device, dtype, stride, T, V, px, pt = _rows(logits, targets)
    # (tensors of their own: views of one could not be changed in place behind an autograd function)
    logprob = torch.empty((T,), dtype=_f32, device=device)
    entropy = torch.empty((T,), dtype=_f32, device=device)
    norm = torch.empty((T, 2), dtype=_f32, device=device)
    rank = torch.empty((T,), dtype=_i32, device=device)
    need = _known_bytes("fp8bs_logprobs_workspace_bytes", T, V, top)
    top_ids = torch.empty((T, top), dtype=_i32, device=device)
    top_logprobs = torch.empty((T, top), dtype=_f32, device=device)
    ws = _workspace(need, device)
    _call("fp8bs_logprobs", device, px, dtype, stride, pt, T, V, top, logprob.data_ptr(), entropy.data_ptr(),
          norm.data_ptr(), rank.data_ptr(), top_ids.data_ptr(), top_logprobs.data_ptr(), ws.data_ptr())
    return logprob, entropy, norm, rank, top_ids, top_logprobs


def fp8bs_logprobs_bwd(logits, targets, norm, entropy, d_logprob, d_entropy):
    """Gradient of fp8bs_logprobs' logprob and entropy (f32 [T] each), with
    norm and entropy as it returned them: d_logits [T][V], contiguous, of logits' dtype."""
    device, dtype, stride, T, V, px, pt = _rows(logits, targets)
    side = [_ptr(t, name, _f32, shape, device) for t, name, shape in
            ((norm, "norm", (T, 2)), (entropy, "entropy", (T,)), (d_logprob, "d_logprob", (T,)), (d_entropy, "d_entropy", (T,)))]
    d_logits = torch.empty((T, V), dtype=logits.dtype, device=device)
    _call("fp8bs_logprobs_bwd", device, px, dtype, stride, pt, *side, T, V, d_logits.data_ptr())
    return d_logits
