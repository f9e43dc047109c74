"""The attention operators' header, exports and host-side refusals (no GPU: every
call below fails validation or has nothing to do)."""

import ctypes
import os
import re

import pytest

import fp8_block_scaled_x1_amd as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, P, MIS = None, 0x10000, 0x10002


def _declared():
    text = open(os.path.join(ROOT, "include", "fp8bs_attn.h")).read()
    return re.findall(r"FP8BS_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fb.LIB_PATH):
        pytest.skip("libfp8bs.so not built")
    return fb.attn_lib()


def test_header_and_exports(L):
    assert set(_declared()) == {
        "fp8bs_mla_prefill", "fp8bs_mla_prefill_workspace_bytes", "fp8bs_mla_prefill_bwd", "fp8bs_mla_prefill_bwd_workspace_bytes", "fp8bs_mla_decode",
        "fp8bs_mla_decode_shared", "fp8bs_mla_decode_workspace_bytes", "fp8bs_verify_drafts",
        "fp8bs_verify_drafts_workspace_bytes", "fp8bs_attn_version"}
    raw = ctypes.CDLL(fb.LIB_PATH)
    for name in _declared():
        assert hasattr(raw, name), name
    assert L.fp8bs_attn_version() == fb.ATTN_VERSION
    assert fb.status_string(-9) == "a scalar argument is outside its range"


def _prefill(L, **kw):
    a = dict(q=P, qs=384, kv=P, kvs=512, r=P, rs=64, cq=P, ck=P, B=2, Tq=10, Tk=12, H=2, scale=0.1, causal=1, out=P,
             lse=P, ws=NULL, stream=NULL)
    a.update(kw)
    return L.fp8bs_mla_prefill(*a.values())


def test_prefill_refusals(L):
    assert _prefill(L, Tq=0, q=NULL, out=NULL) == 0
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-2), dict(H=0), dict(B=0), dict(qs=376), dict(kvs=504), dict(rs=56)):
        assert _prefill(L, **kw) == -2, kw
    for kw in (dict(qs=388), dict(kvs=517), dict(rs=65), dict(q=MIS), dict(kv=MIS), dict(r=P + 8), dict(out=MIS),
               dict(cq=P + 1), dict(lse=MIS)):
        assert _prefill(L, **kw) == -3, kw
    for name in ("q", "kv", "r", "cq", "ck", "out", "lse"):
        assert _prefill(L, **{name: NULL}) == -1, name
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert _prefill(L, scale=s) == -9
    assert _prefill(L, Tq=1 << 31) == -7
    assert _prefill(L, H=70000, qs=70000 * 192, kvs=70000 * 256) == -7


def test_prefill_workspace(L):
    ws = L.fp8bs_mla_prefill_workspace_bytes
    assert ws(-1, 1, 1, 1) == -2 and ws(1, 1, 1, 0) == -2 and ws(1, 1 << 31, 1, 1) == -7
    assert ws(2, 300, 300, 16) == 0 and ws(0, 0, 0, 4) == 0          # few keys: nothing to share
    assert ws(2, 40000, 40000, 128) == 0                             # more than enough blocks
    # few queries, many keys: whole parts of [Tq][H] rows of 128 numbers, a maximum and a sum
    n = ws(1, 20, 50000, 4)
    assert n > 0 and n % (20 * 4 * 130 * 4) == 0 and n // (20 * 4 * 130 * 4) >= 2
    many = dict(B=1, Tq=20, Tk=50000, H=4, qs=768, kvs=1024)
    assert _prefill(L, **many, ws=NULL) == -1 and _prefill(L, **many, ws=P + 8) == -3


def test_prefill_workspace_of_filled_devices(L):
    # Blocks of 256 queries, which are not cut in parts, from one and a half per compute unit on: counted for requests
    # of average length, not with one more for each of them.
    ws = L.fp8bs_mla_prefill_workspace_bytes
    assert ws(1, 4200, 34200, 32) == 0                               # 17 blocks on 32 heads
    assert ws(1, 2300, 32300, 32) > 0                                # 9 blocks
    # one block of 128 holds a request's queries: parts where the device's last turn would be a short one
    assert ws(5, 5, 5 * 30001, 128) > 0 and ws(7, 7, 7 * 20001, 128) > 0
    assert ws(8, 8, 8 * 20001, 128) == 0                             # whole turns
    # the workspace stays bounded
    assert ws(1 << 20, 1 << 20, (1 << 31) - 1, 8) == 0


def test_prefill_bwd_refusals(L):
    def call(**kw):
        a = dict(dout=P, q=P, qs=384, kv=P, kvs=512, r=P, rs=64, out=P, lse=P, cq=P, ck=P, B=2, Tq=10, Tk=12, H=2,
                 scale=0.1, causal=1, dq=P, dkv=P, dr=P, ws=P, stream=NULL)
        a.update(kw)
        return L.fp8bs_mla_prefill_bwd(*a.values())
    assert call(Tq=0, Tk=0, ws=NULL) == 0
    for name in ("dout", "q", "kv", "r", "out", "lse", "cq", "ck", "dq", "dkv", "dr", "ws"):
        assert call(**{name: NULL}) == -1, name
    for name in ("dout", "out", "dq", "dkv", "dr", "ws"):
        assert call(**{name: P + 8}) == -3, name
    assert call(scale=0.0) == -9 and call(H=0) == -2
    ws = L.fp8bs_mla_prefill_bwd_workspace_bytes
    assert ws(10, 12, 2) == 2 * 256 + 12 * 2 * 64 * 4 and ws(-1, 2, 2) == -2 and ws(4, 4, 0) == -2


def _decode(L, shared=False, **kw):
    a = dict(q=P, kind=0, cache=P, sc=P, rope=P, pages=9, page=16)
    if shared:
        a.update(pt=P, pp=3, pl=P)
    a.update(table=P, width=4, lens=P, B=2, T=1, H=4, scale=0.1, out=P, lse=P, ws=P, stream=NULL)
    a.update(kw)
    return (L.fp8bs_mla_decode_shared if shared else L.fp8bs_mla_decode)(*a.values())


@pytest.mark.parametrize("shared", [False, True])
def test_decode_refusals(L, shared):
    assert _decode(L, shared, B=0, q=NULL) == 0
    for kw in (dict(B=-1), dict(T=0), dict(H=0), dict(page=0), dict(width=-1), dict(pages=-1), dict(pages=0)):
        assert _decode(L, shared, **kw) == -2, kw
    assert _decode(L, shared, kind=2) == -5
    for name in ("q", "cache", "table", "lens", "out", "lse", "ws") + (("pt", "pl") if shared else ()):
        assert _decode(L, shared, **{name: NULL}) == -1, name
    assert _decode(L, shared, kind=1, sc=NULL) == -1 and _decode(L, shared, kind=1, rope=NULL) == -1
    for name in ("q", "cache", "out", "ws"):
        assert _decode(L, shared, **{name: P + 8}) == -3, name
    for name in ("table", "lens", "lse"):
        assert _decode(L, shared, **{name: MIS}) == -3, name
    assert _decode(L, shared, kind=1, sc=P + 4) == -3
    assert _decode(L, shared, scale=0.0) == -9
    assert _decode(L, shared, width=1 << 28) == -7          # more tokens than an int32 length says
    assert _decode(L, shared, H=1 << 24) == -7


def test_decode_workspace(L):
    ws = L.fp8bs_mla_decode_workspace_bytes
    assert ws(2, 0, 4, 4, 16, 0) == -2 and ws(2, 1, 4, 4, 0, 0) == -2 and ws(2, 1, 4, 4, 16, -1) == -2
    assert 0 < ws(2, 1, 4, 4, 16, 0) < ws(2, 1, 4, 4, 16, 3)


def test_verify_refusals(L):
    def call(**kw):
        a = dict(p=P, q=P, dtype=0, d=P, n=P, u=P, un=P, B=3, K=2, V=100, t=P, a=P, ws=P, stream=NULL)
        a.update(kw)
        return L.fp8bs_verify_drafts(*a.values())
    assert call(B=0, p=NULL) == 0
    assert call(dtype=2) == -4
    for kw in (dict(K=-1), dict(K=64), dict(B=-1), dict(V=0)):
        assert call(**kw) == -2, kw
    assert call(V=(1 << 24) + 1) == -7
    for name in ("p", "d", "n", "u", "un", "t", "a", "ws"):
        assert call(**{name: NULL}) == -1, name
    for name in ("p", "q", "d", "n", "u", "un", "t", "a"):
        assert call(**{name: MIS}) == -3, name
    assert call(ws=P + 4) == -3
    assert L.fp8bs_verify_drafts_workspace_bytes(2, 8193) == 16 * 2 * 3


def test_attention_beyond_what_a_launch_holds(L):
    # refused by its sizes, before a first kernel is enqueued: a launch has fewer than 2^32 threads
    many = dict(B=65536, Tq=65536, Tk=65536, H=128, qs=128 * 192, kvs=128 * 256)
    assert _prefill(L, **many) == -7
    bwd = dict(dout=P, q=P, qs=128 * 192, kv=P, kvs=128 * 256, r=P, rs=64, out=P, lse=P, cq=P, ck=P, B=65536, Tq=65536,
               Tk=65536, H=128, scale=0.1, causal=1, dq=P, dkv=P, dr=P, ws=P, stream=NULL)
    assert L.fp8bs_mla_prefill_bwd(*bwd.values()) == -7
    bwd.update(B=1, Tq=1, Tk=1 << 26, H=1, qs=192, kvs=256)          # the rotary sum: 64 threads a key
    assert L.fp8bs_mla_prefill_bwd(*bwd.values()) == -7
    # the join of the pieces: a wave a row
    for shared in (False, True):
        assert _decode(L, shared, B=1 << 16, T=8, H=128) == -7
    ws = L.fp8bs_mla_decode_workspace_bytes
    assert ws(1 << 16, 8, 128, 4, 16, 0) == -7 and ws((1 << 26) - 1, 1, 1, 1, 1, 0) == -7 and ws((1 << 16) - 1, 8, 128, 4, 16, 0) > 0


def test_verify_more_requests_than_a_launch_holds(L):
    # one workgroup of 256 threads per request and chunk, and a launch has fewer than 2^32 threads
    ws = L.fp8bs_verify_drafts_workspace_bytes
    assert ws((1 << 24) - 1, 1) == 16 * 2 * ((1 << 24) - 1)
    assert ws((1 << 23) - 1, 8193) == 16 * 3 * ((1 << 23) - 1)
    for B, V in ((1 << 24, 1), (1 << 23, 8193), (1 << 27, 1), (1 << 28, 1), ((1 << 31) - 1, 1), (1 << 13, 1 << 24)):
        assert ws(B, V) == -7, (B, V)
        assert L.fp8bs_verify_drafts(P, NULL, 0, NULL, P, NULL, P, B, 0, V, P, P, P, NULL) == -7, (B, V)


def test_binding_refusals():
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    q, kv, kr, cu = torch.zeros(4, 2, 192, dtype=bf), torch.zeros(4, 2, 256, dtype=bf), torch.zeros(4, 64, dtype=bf), \
        torch.tensor([0, 4], dtype=i32)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_mla_prefill(q, kv, kr, cu, cu, 0.1)
    with pytest.raises(ValueError, match="q must be"):
        fb.fp8bs_mla_prefill(q[..., :128], kv, kr, cu, cu, 0.1)
    with pytest.raises(ValueError, match="q must be"):
        fb.fp8bs_mla_decode(q, kv, cu[None], cu, 0.1)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_mla_decode(q.new_zeros(1, 1, 4, 576), q.new_zeros(3, 16, 576), cu[None], cu, 0.1)
    with pytest.raises(TypeError, match="torch tensor"):
        fb.fp8bs_mla_decode_shared([1], q, cu, cu, cu[None], cu, 0.1)
    with pytest.raises(ValueError, match="p must be"):
        fb.fp8bs_verify_drafts(torch.zeros(4, 5), None, cu, cu, cu, cu)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_verify_drafts(torch.zeros(1, 2, 5), None, cu, cu, cu, cu)
    with pytest.raises(TypeError, match="one dtype"):
        fb.fp8bs_verify_drafts(torch.zeros(1, 2, 5), torch.zeros(1, 1, 5, dtype=bf), cu, cu, cu, cu)
