"""ctypes binding of the attention and draft-verification operators
(include/fp8bs_attn.h): argument marshalling only, as in _lib.

Every function has the name of the C entry point it calls, checks the tensors
it is given, allocates the outputs and the workspace with torch and calls the
library on the current torch stream of the inputs' device. Results carry no
autograd graph, whatever their inputs require: fp8bs_mla_prefill_bwd gives the
gradients (examples/latent_attention.py wraps the two in an autograd function).
"""

import ctypes
import functools

import torch

from . import _lib

ATTN_VERSION = 1
CACHE_BF16, CACHE_FP8 = 0, 1

_i, _i64, _f, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p

_SIGNATURES = {
    "fp8bs_mla_prefill": [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i, _i64, _i64, _i, _f, _i, _vp, _vp, _vp, _vp],
    "fp8bs_mla_prefill_workspace_bytes": [_i, _i64, _i64, _i],
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


_bf16, _f32, _i32, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _ptr(t, name, dtype, shape, device):
    """The address of a contiguous tensor of this dtype, shape and device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on_gpu(t, name, dims):
    """The device of the tensor that the call goes by, after its first checks."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    shape, fits = t.shape, t.dim() == len(dims)
    if fits:
        for d, n in zip(dims, shape):      # (a generator costs 0.4 us more)
            fits = fits and (d is None or d == n)
    if not fits:
        raise ValueError(f"{name} must be [{']['.join('*' if d is None else str(d) for d in dims)}], got {tuple(shape)}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    return t.device


def _tokens(t, name, inner, device):
    """(pointer, numbers from token to token) of a BF16 tensor [T][inner...]
    whose tokens are contiguous inside but may lie apart."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape[1:] != inner:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (tokens, {', '.join(map(str, inner))})")
    if t.dtype != _bf16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {_bf16}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    n = 1
    if t.is_contiguous():
        for size in inner:
            n *= size
        return t.data_ptr(), n
    for size, stride in zip(reversed(inner), reversed(t.stride()[1:])):
        if size != 1 and stride != n:
            raise ValueError(f"{name}: the numbers of a token must be contiguous")
        n *= size
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else n


# the current stream's handle without the Stream object around it (2 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, device, *args):
    """Calls the entry point on the device's current stream, with the device current."""
    entry, index = getattr(attn_lib(), fn), device.index
    if index == torch.cuda.current_device():
        status = entry(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = entry(*args, _raw_stream(index))
    if status != 0:
        raise _lib.Fp8bsError(fn, status)


def _bytes(fn, *sizes):
    """What a *_workspace_bytes function says of these sizes."""
    n = getattr(attn_lib(), fn)(*sizes)
    if n < 0:
        raise _lib.Fp8bsError(fn, n)
    return n


@functools.lru_cache(maxsize=4096)
def _bytes_on(device_index, fn, *sizes):
    """The same where the answer depends on the device: asked once per device and sizes."""
    with torch.cuda.device(device_index):
        return _bytes(fn, *sizes)


def _workspace(need, device):
    return torch.empty(max(need, 16), dtype=_u8, device=device)


def _prefill_args(q, kv, k_rope, cu_q, cu_k):
    device = _on_gpu(q, "q", (None, None, 192))
    H = q.shape[1]
    pq, sq = _tokens(q, "q", (H, 192), device)
    pkv, skv = _tokens(kv, "kv", (H, 256), device)
    pr, sr = _tokens(k_rope, "k_rope", (64,), device)
    if k_rope.shape[0] != kv.shape[0]:
        raise ValueError("kv and k_rope disagree on the number of tokens")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must have B+1 entries")
    off = cu_q.shape
    return device, (pq, sq, pkv, skv, pr, sr), (_ptr(cu_q, "cu_q", _i32, off, device),
                                                _ptr(cu_k, "cu_k", _i32, off, device), off[0] - 1, q.shape[0],
                                                kv.shape[0], H)


def fp8bs_mla_prefill(q, kv, k_rope, cu_q, cu_k, scale, causal=True):
    """Latent attention, expanded form, of packed requests: q [Tq][H][192], kv
    [Tk][H][256] (keys then values of each head), k_rope [Tk][64], all BF16 and
    possibly with gaps between tokens; cu_q, cu_k int32 [B+1] on the GPU.
    Returns (out bf16 [Tq][H][128], lse f32 [H][Tq])."""
    device, ptrs, sizes = _prefill_args(q, kv, k_rope, cu_q, cu_k)
    Tq, H = q.shape[:2]
    out = torch.empty((Tq, H, 128), dtype=_bf16, device=device)
    lse = torch.empty((H, Tq), dtype=_f32, device=device)
    need = _bytes("fp8bs_mla_prefill_workspace_bytes", *sizes[2:])
    ws = torch.empty(need, dtype=_u8, device=device) if need else None
    _call("fp8bs_mla_prefill", device, *ptrs, *sizes, float(scale), int(bool(causal)), out.data_ptr(), lse.data_ptr(),
          ws.data_ptr() if need else None)
    return out, lse


def fp8bs_mla_prefill_bwd(dout, q, kv, k_rope, out, lse, cu_q, cu_k, scale, causal=True):
    """Gradients of fp8bs_mla_prefill's out: (dq [Tq][H][192], dkv [Tk][H][256],
    dk_rope [Tk][64]), BF16; out and lse as the forward returned them."""
    device, ptrs, sizes = _prefill_args(q, kv, k_rope, cu_q, cu_k)
    Tq, H = q.shape[:2]
    Tk = kv.shape[0]
    pd, po = _ptr(dout, "dout", _bf16, (Tq, H, 128), device), _ptr(out, "out", _bf16, (Tq, H, 128), device)
    pl = _ptr(lse, "lse", _f32, (H, Tq), device)
    ws = _workspace(_bytes("fp8bs_mla_prefill_bwd_workspace_bytes", Tq, Tk, H), device)
    dq = torch.empty((Tq, H, 192), dtype=_bf16, device=device)
    dkv = torch.empty((Tk, H, 256), dtype=_bf16, device=device)
    dk_rope = torch.empty((Tk, 64), dtype=_bf16, device=device)
    _call("fp8bs_mla_prefill_bwd", device, pd, *ptrs, po, pl, *sizes, float(scale), int(bool(causal)), dq.data_ptr(),
          dkv.data_ptr(), dk_rope.data_ptr(), ws.data_ptr())
    return dq, dkv, dk_rope


def _cache_args(cache, device):
    """(kind, pointers, pages, page size) of a cache: BF16 [pages][page][576],
    or the FP8 triple (codes uint8 [..][512], scales f32 [..][4], rope bf16 [..][64])."""
    if isinstance(cache, (tuple, list)):
        if len(cache) != 3:
            raise ValueError("an FP8 cache is (codes, scales, rope)")
        codes, scales, rope = cache
        if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
            raise ValueError("cache codes must be [pages][page][512]")
        n, page = codes.shape[:2]
        return (CACHE_FP8, _ptr(codes, "cache codes", _u8, (n, page, 512), device),
                _ptr(scales, "cache scales", _f32, (n, page, 4), device),
                _ptr(rope, "cache rope", _bf16, (n, page, 64), device), n, page)
    if not isinstance(cache, torch.Tensor) or cache.dim() != 3:
        raise ValueError("cache must be [pages][page][576] or (codes, scales, rope)")
    n, page = cache.shape[:2]
    return CACHE_BF16, _ptr(cache, "cache", _bf16, (n, page, 576), device), None, None, n, page


def _decode(fn, q, cache, prefix, table, lens, scale):
    device = _on_gpu(q, "q", (None, None, None, 576))
    B, T, H, _ = q.shape
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be [B][width]")
    width = table.shape[1]
    pq = _ptr(q, "q", _bf16, q.shape, device)
    cache_args = _cache_args(cache, device)
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
    ws = _workspace(_bytes_on(device.index, "fp8bs_mla_decode_workspace_bytes", B, T, H, width, cache_args[5], n_pre), device)
    _call(fn, device, pq, *cache_args, *pre, pt, width, pl, B, T, H, float(scale), out.data_ptr(), lse.data_ptr(),
          ws.data_ptr())
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
    if isinstance(q, torch.Tensor) and isinstance(p, torch.Tensor) and q.dtype != p.dtype:
        raise TypeError("p and q must have one dtype")
    device = _on_gpu(p, "p", (None, None, None))
    B, K1, V = p.shape
    K = K1 - 1
    if K < 0:
        raise ValueError("p must be [B][K+1][V]")
    dtype = p.dtype
    if dtype not in (_f32, _bf16):
        raise TypeError(f"p has dtype {dtype}, expected float32 or bfloat16")
    pp = _ptr(p, "p", dtype, p.shape, device)
    pq = None if q is None else _ptr(q, "q", dtype, (B, K, V), device)
    args = (_ptr(drafts, "drafts", _i32, (B, K), device), _ptr(n_drafts, "n_drafts", _i32, (B,), device),
            _ptr(u, "u", _f32, (B, K), device), _ptr(u_next, "u_next", _f32, (B,), device))
    tokens = torch.empty((B, K1), dtype=_i32, device=device)
    accepted = torch.empty((B,), dtype=_i32, device=device)
    ws = _workspace(_bytes("fp8bs_verify_drafts_workspace_bytes", B, V), device)
    _call("fp8bs_verify_drafts", device, pp, pq, _lib.BF16 if dtype == _bf16 else _lib.F32, *args, B, K, V,
          tokens.data_ptr(), accepted.data_ptr(), ws.data_ptr())
    return tokens, accepted
