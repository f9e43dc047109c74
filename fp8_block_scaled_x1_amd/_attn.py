"""ctypes binding of the attention and draft-verification operators
(include/fp8bs_attn.h): argument marshalling only, as in _lib.

Every function has the name of the C entry point it calls, checks the tensors
it is given, allocates the outputs and the workspace with torch and calls the
library on the current torch stream of the inputs' device.
"""

import ctypes

import torch

from . import _lib
from ._lib import _check, _dev, _in_dtype, _stream

ATTN_VERSION = 1
CACHE_BF16, CACHE_FP8 = 0, 1

_i, _i64, _f, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p

_SIGNATURES = {
    "fp8bs_mla_prefill": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i, _i64, _i64, _i, _f, _i, _vp, _vp, _vp],
    "fp8bs_mla_prefill_bwd": [_vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i, _i64, _i64, _i, _f, _i,
                              _vp, _vp, _vp, _vp, _vp],
    "fp8bs_mla_prefill_bwd_workspace_bytes": [_i64, _i64, _i],
    "fp8bs_mla_decode": [_vp, _i, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _i, _i, _i, _f, _vp, _vp, _vp, _vp],
    "fp8bs_mla_decode_shared": [_vp, _i, _vp, _vp, _vp, _i64, _i, _vp, _i64, _vp, _vp, _i64, _vp, _i, _i, _i, _f, _vp,
                                _vp, _vp, _vp],
    "fp8bs_mla_decode_workspace_bytes": [_i, _i, _i, _i64, _i, _i64],
    "fp8bs_verify_drafts": [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i64, _vp, _vp, _vp, _vp],
    "fp8bs_verify_drafts_workspace_bytes": [_i, _i64],
    "fp8bs_attn_version": [],
}

_attn = None


def attn_lib():
    """The loaded library with the signatures of fp8bs_attn.h."""
    global _attn
    if _attn is None:
        handle = _lib.lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = _i64 if name.endswith("_bytes") else _i
        if handle.fp8bs_attn_version() != ATTN_VERSION:
            raise ImportError(f"libfp8bs attention version {handle.fp8bs_attn_version()} != {ATTN_VERSION}")
        _attn = handle
    return _attn


_BF16, _F32, _I32, _U8 = (torch.bfloat16,), (torch.float32,), (torch.int32,), (torch.uint8,)


def _want(t, name, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _same_device(**tensors):
    devs = {t.device for t in tensors.values() if t is not None}
    if len(devs) > 1:
        raise ValueError(f"{', '.join(tensors)} are on different devices")


def _tokens(t, name, inner):
    """(pointer, numbers from token to token) of a BF16 tensor [T][inner...]
    whose tokens are contiguous inside but may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if tuple(t.shape[1:]) != tuple(inner) or t.dim() != 1 + len(inner):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (tokens, {', '.join(map(str, inner))})")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    n = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != n:
            raise ValueError(f"{name}: the numbers of a token must be contiguous")
        n *= size
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else n


def _workspace(nbytes, fn, device):
    _check(fn, min(0, nbytes))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _prefill_args(q, kv, k_rope, cu_q, cu_k):
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be [Tq][H][192]")
    H = q.shape[1]
    pq, sq = _tokens(q, "q", (H, 192))
    pkv, skv = _tokens(kv, "kv", (H, 256))
    pr, sr = _tokens(k_rope, "k_rope", (64,))
    if k_rope.shape[0] != kv.shape[0]:
        raise ValueError("kv and k_rope disagree on the number of tokens")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must have B+1 entries")
    _want(cu_k, "cu_k", cu_q.shape)
    _same_device(q=q, kv=kv, k_rope=k_rope, cu_q=cu_q, cu_k=cu_k)
    return (pq, sq, pkv, skv, pr, sr), (_dev(cu_q, "cu_q", _I32), _dev(cu_k, "cu_k", _I32), cu_q.shape[0] - 1,
                                        q.shape[0], kv.shape[0], H)


def fp8bs_mla_prefill(q, kv, k_rope, cu_q, cu_k, scale, causal=True):
    """Latent attention, expanded form, of packed requests: q [Tq][H][192], kv
    [Tk][H][256] (keys then values of each head), k_rope [Tk][64], all BF16 and
    possibly with gaps between tokens; cu_q, cu_k int32 [B+1] on the GPU.
    Returns (out bf16 [Tq][H][128], lse f32 [H][Tq])."""
    ptrs, sizes = _prefill_args(q, kv, k_rope, cu_q, cu_k)
    Tq, H = q.shape[:2]
    out = torch.empty((Tq, H, 128), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((H, Tq), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        _check("fp8bs_mla_prefill", attn_lib().fp8bs_mla_prefill(*ptrs, *sizes, float(scale), int(bool(causal)),
                                                                 out.data_ptr(), lse.data_ptr(), _stream(q)))
    return out, lse


def fp8bs_mla_prefill_bwd(dout, q, kv, k_rope, out, lse, cu_q, cu_k, scale, causal=True):
    """Gradients of fp8bs_mla_prefill's out: (dq [Tq][H][192], dkv [Tk][H][256],
    dk_rope [Tk][64]), BF16; out and lse as the forward returned them."""
    ptrs, sizes = _prefill_args(q, kv, k_rope, cu_q, cu_k)
    Tq, H = q.shape[:2]
    Tk = kv.shape[0]
    _want(dout, "dout", (Tq, H, 128))
    _want(out, "out", (Tq, H, 128))
    _want(lse, "lse", (H, Tq))
    _same_device(q=q, dout=dout, out=out, lse=lse)
    pd, po, pl = _dev(dout, "dout", _BF16), _dev(out, "out", _BF16), _dev(lse, "lse", _F32)
    L = attn_lib()
    ws = _workspace(L.fp8bs_mla_prefill_bwd_workspace_bytes(Tq, Tk, H), "fp8bs_mla_prefill_bwd_workspace_bytes", q.device)
    dq = torch.empty((Tq, H, 192), dtype=torch.bfloat16, device=q.device)
    dkv = torch.empty((Tk, H, 256), dtype=torch.bfloat16, device=q.device)
    dk_rope = torch.empty((Tk, 64), dtype=torch.bfloat16, device=q.device)
    with torch.cuda.device(q.device):
        _check("fp8bs_mla_prefill_bwd",
               L.fp8bs_mla_prefill_bwd(pd, *ptrs, po, pl, *sizes, float(scale), int(bool(causal)), dq.data_ptr(),
                                       dkv.data_ptr(), dk_rope.data_ptr(), ws.data_ptr(), _stream(q)))
    return dq, dkv, dk_rope


def _cache_args(cache):
    """(kind, pointers, pages, page size) of a cache: BF16 [pages][page][576],
    or the FP8 triple (codes uint8 [..][512], scales f32 [..][4], rope bf16 [..][64])."""
    if isinstance(cache, (tuple, list)):
        if len(cache) != 3:
            raise ValueError("an FP8 cache is (codes, scales, rope)")
        codes, scales, rope = cache
        if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
            raise ValueError("cache codes must be [pages][page][512]")
        pages, page = codes.shape[:2]
        _want(codes, "cache codes", (pages, page, 512))
        _want(scales, "cache scales", (pages, page, 4))
        _want(rope, "cache rope", (pages, page, 64))
        _same_device(codes=codes, scales=scales, rope=rope)
        return (CACHE_FP8, _dev(codes, "cache codes", _U8), _dev(scales, "cache scales", _F32),
                _dev(rope, "cache rope", _BF16), pages, page), codes
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3:
        raise ValueError("cache must be [pages][page][576] or (codes, scales, rope)")
    pages, page = cache.shape[:2]
    _want(cache, "cache", (pages, page, 576))
    return (CACHE_BF16, _dev(cache, "cache", _BF16), None, None, pages, page), cache


def _decode(fn, q, cache, prefix, table, lens, scale):
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != 576:
        raise ValueError("q must be [B][T][H][576]")
    B, T, H, _ = q.shape
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be [B][width]")
    _want(lens, "lens", (B,))
    cache_args, first = _cache_args(cache)
    page = cache_args[-1]
    width = table.shape[1]
    pre, n_pre = (), 0
    if prefix is not None:
        prefix_table, prefix_len = prefix
        if not isinstance(prefix_table, torch.Tensor) or prefix_table.dim() != 1:
            raise ValueError("prefix_table must be [pages of the prefix]")
        _want(prefix_len, "prefix_len", (1,))
        _same_device(q=q, prefix_table=prefix_table, prefix_len=prefix_len)
        n_pre = prefix_table.shape[0]
        pre = (_dev(prefix_table, "prefix_table", _I32), n_pre, _dev(prefix_len, "prefix_len", _I32))
    _same_device(q=q, cache=first, table=table, lens=lens)
    pq, pt, pl = _dev(q, "q", _BF16), _dev(table, "table", _I32), _dev(lens, "lens", _I32)
    L = attn_lib()
    out = torch.empty((B, T, H, 512), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        ws = _workspace(L.fp8bs_mla_decode_workspace_bytes(B, T, H, width, page, n_pre),
                        "fp8bs_mla_decode_workspace_bytes", q.device)
        _check(fn, getattr(L, fn)(pq, *cache_args, *pre, pt, width, pl, B, T, H, float(scale), out.data_ptr(),
                                  lse.data_ptr(), ws.data_ptr(), _stream(q)))
    return out, lse


def fp8bs_mla_decode(q, cache, table, lens, scale):
    """Latent attention, absorbed form, over a paged cache: q [B][T][H][576] BF16,
    cache BF16 [pages][page][576] or FP8 (codes, scales, rope), table int32
    [B][width], lens int32 [B]. Returns (out bf16 [B][T][H][512], lse f32 [B][T][H])."""
    return _decode("fp8bs_mla_decode", q, cache, None, table, lens, scale)


def fp8bs_mla_decode_shared(q, cache, prefix_table, prefix_len, table, lens, scale):
    """fp8bs_mla_decode for requests that share a prefix of prefix_len[0] tokens
    in the pages prefix_table; table and lens hold each request's own tokens."""
    return _decode("fp8bs_mla_decode_shared", q, cache, (prefix_table, prefix_len), table, lens, scale)


def fp8bs_verify_drafts(p, q, drafts, n_drafts, u, u_next):
    """Acceptance of drafted tokens and the token after them: p [B][K+1][V] and q
    [B][K][V] (or None: drafts chosen without chance) probabilities, f32 or bf16;
    drafts int32 [B][K], n_drafts int32 [B], u f32 [B][K], u_next f32 [B].
    Returns (tokens int32 [B][K+1], accepted int32 [B])."""
    if not isinstance(p, torch.Tensor) or p.dim() != 3:
        raise ValueError("p must be [B][K+1][V]")
    B, K, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    if K < 0:
        raise ValueError("p must be [B][K+1][V]")
    if q is not None:
        _want(q, "q", (B, K, V))
        if q.dtype != p.dtype:
            raise TypeError("p and q must have one dtype")
    pp, pq = _dev(p, "p", (torch.float32, torch.bfloat16)), None
    if q is not None:
        pq = _dev(q, "q", (torch.float32, torch.bfloat16))
    _want(drafts, "drafts", (B, K))
    _want(n_drafts, "n_drafts", (B,))
    _want(u, "u", (B, K))
    _want(u_next, "u_next", (B,))
    _same_device(p=p, q=q, drafts=drafts, n_drafts=n_drafts, u=u, u_next=u_next)
    args = (_dev(drafts, "drafts", _I32), _dev(n_drafts, "n_drafts", _I32), _dev(u, "u", _F32),
            _dev(u_next, "u_next", _F32))
    L = attn_lib()
    tokens = torch.empty((B, K + 1), dtype=torch.int32, device=p.device)
    accepted = torch.empty((B,), dtype=torch.int32, device=p.device)
    ws = _workspace(L.fp8bs_verify_drafts_workspace_bytes(B, V), "fp8bs_verify_drafts_workspace_bytes", p.device)
    with torch.cuda.device(p.device):
        _check("fp8bs_verify_drafts",
               L.fp8bs_verify_drafts(pp, pq, _in_dtype(p), *args, B, K, V, tokens.data_ptr(), accepted.data_ptr(),
                                     ws.data_ptr(), _stream(p)))
    return tokens, accepted
