"""The serving operators' header, exports and host-side refusals (no GPU: every
call below fails validation or has nothing to do)."""

import ctypes
import os
import re

import pytest

import fp8_block_scaled_x1_amd as fb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, P, MIS = None, 0x10000, 0x10002


def _declared():
    text = open(os.path.join(ROOT, "include", "fp8bs_serve.h")).read()
    return re.findall(r"FP8BS_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(fb.LIB_PATH):
        pytest.skip("libfp8bs.so not built")
    return fb.serve_lib()


def test_header_and_exports(L):
    assert set(_declared()) == {
        "fp8bs_mla_cache_write", "fp8bs_mla_cache_read", "fp8bs_mla_decode_fp4", "fp8bs_mla_decode_fp4_shared",
        "fp8bs_mla_decode_fp4_workspace_bytes", "fp8bs_moe_tokens", "fp8bs_moe_tokens_workspace_bytes", "fp8bs_logprobs",
        "fp8bs_logprobs_workspace_bytes", "fp8bs_logprobs_bwd", "fp8bs_serve_version"}
    raw = ctypes.CDLL(fb.LIB_PATH)
    for name in _declared():
        assert hasattr(raw, name), name
    assert L.fp8bs_serve_version() == fb.SERVE_VERSION == 1
    text = open(os.path.join(ROOT, "include", "fp8bs_serve.h")).read()
    assert f"#define FP8BS_CACHE_FP4 {fb.CACHE_FP4}\n" in text and "#define FP8BS_SERVE_VERSION 1\n" in text


def _cache(L, read, **kw):
    rows = dict(lat=P, ls=512, rope=P, rs=64)
    pool = dict(kind=2, cache=P, sc=P, cr=P, pages=9, page=16)
    req = dict(table=P, width=4, lens=P)
    if read:
        a = {**pool, **req, "cu": P, "B": 2, "T": 5, **rows}
    else:
        a = {**rows, "cu": P, "B": 2, "T": 5, **pool, **req}
    a.update(stream=NULL)
    a.update(kw)
    return (L.fp8bs_mla_cache_read if read else L.fp8bs_mla_cache_write)(*a.values())


@pytest.mark.parametrize("read", [False, True])
def test_cache_refusals(L, read):
    assert _cache(L, read, T=0, lat=NULL) == 0 and _cache(L, read, B=0, cu=NULL) == 0
    for kind in (-1, 3):
        assert _cache(L, read, kind=kind) == -5
    for kw in (dict(B=-1), dict(T=-1), dict(pages=-1), dict(pages=0), dict(page=0), dict(width=-1), dict(ls=504), dict(rs=56)):
        assert _cache(L, read, **kw) == -2, kw
    for kw in (dict(ls=515), dict(rs=65), dict(lat=MIS), dict(rope=P + 8), dict(cache=P + 8), dict(sc=P + 4), dict(cr=MIS),
               dict(cu=MIS), dict(table=MIS), dict(lens=P + 1)):
        assert _cache(L, read, **kw) == -3, kw
    for name in ("lat", "rope", "cu", "lens", "table", "cache", "sc", "cr"):
        assert _cache(L, read, **{name: NULL}) == -1, name
    for kw in (dict(pages=1 << 31), dict(pages=1 << 28), dict(width=1 << 28), dict(T=(1 << 31) - 8), dict(B=1 << 30),
               dict(ls=1 << 31), dict(rs=1 << 31), dict(T=1 << 28)):
        assert _cache(L, read, **kw) == -7, kw


def test_write_without_a_table_has_nothing_to_do(L):
    assert _cache(L, False, width=0, table=NULL, cache=NULL) == 0


def _decode(L, shared=False, **kw):
    a = dict(q=P, cache=P, sc=P, rope=P, pages=9, page=16)
    if shared:
        a.update(pt=P, pp=3, pl=P)
    a.update(table=P, width=4, lens=P, B=2, T=1, H=4, scale=0.1, out=P, lse=P, ws=P, stream=NULL)
    a.update(kw)
    return (L.fp8bs_mla_decode_fp4_shared if shared else L.fp8bs_mla_decode_fp4)(*a.values())


@pytest.mark.parametrize("shared", [False, True])
def test_decode_refusals(L, shared):
    assert _decode(L, shared, B=0, q=NULL) == 0
    for kw in (dict(B=-1), dict(T=0), dict(H=0), dict(page=0), dict(width=-1), dict(pages=-1), dict(pages=0)):
        assert _decode(L, shared, **kw) == -2, kw
    for name in ("q", "cache", "sc", "rope", "table", "lens", "out", "lse", "ws") + (("pt", "pl") if shared else ()):
        assert _decode(L, shared, **{name: NULL}) == -1, name
    for name in ("q", "cache", "sc", "rope", "out", "ws"):
        assert _decode(L, shared, **{name: P + 8}) == -3, name
    for name in ("table", "lens", "lse") + (("pt", "pl") if shared else ()):
        assert _decode(L, shared, **{name: MIS}) == -3, name
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert _decode(L, shared, scale=s) == -9
    for kw in (dict(width=1 << 28), dict(H=1 << 24), dict(pages=1 << 28), dict(B=1 << 16, T=8, H=128)):
        assert _decode(L, shared, **kw) == -7, kw


def test_decode_workspace(L):
    ws = L.fp8bs_mla_decode_fp4_workspace_bytes
    assert ws(2, 0, 4, 4, 16, 0) == -2 and ws(2, 1, 4, 4, 0, 0) == -2 and ws(2, 1, 4, 4, 16, -1) == -2
    assert 0 < ws(2, 1, 4, 4, 16, 0) < ws(2, 1, 4, 4, 16, 3)
    assert ws(1 << 16, 8, 128, 4, 16, 0) == -7


def test_moe_refusals(L):
    def call(**kw):
        a = dict(x=P, T=5, K=256, ids=P, w=P, topk=2, wu=P, su=P, wd=P, sd=P, E=8, F=128, out=P, ws=P, stream=NULL)
        a.update(kw)
        return L.fp8bs_moe_tokens(*a.values())
    assert call(T=0, x=NULL) == 0
    for kw in (dict(T=-1), dict(T=65), dict(topk=0), dict(topk=65), dict(E=0), dict(E=1025), dict(K=0), dict(K=200),
               dict(F=0), dict(F=64)):
        assert call(**kw) == -2, kw
    assert call(K=(1 << 16) + 128) == -7 and call(F=(1 << 16) + 128) == -7
    for name in ("x", "ids", "w", "wu", "su", "wd", "sd", "out", "ws"):
        assert call(**{name: NULL}) == -1, name
    for name in ("x", "wu", "wd", "out", "ws"):
        assert call(**{name: P + 8}) == -3, name
    for name in ("ids", "w", "su", "sd"):
        assert call(**{name: MIS}) == -3, name
    ws = L.fp8bs_moe_tokens_workspace_bytes
    assert ws(5, 2, 256, 128) >= 2 * 5 * 2 * 128 and ws(65, 2, 256, 128) == -2 and ws(5, 2, 100, 128) == -2 and ws(5, 2, 256, 1 << 17) == -7


def test_logprobs_refusals(L):
    def call(**kw):
        a = dict(x=P, dtype=0, stride=100, y=P, T=3, V=100, top=5, lp=P, h=P, norm=P, rank=P, ti=P, tl=P, ws=P, stream=NULL)
        a.update(kw)
        return L.fp8bs_logprobs(*a.values())

    def back(**kw):
        a = dict(x=P, dtype=0, stride=100, y=P, norm=P, h=P, dl=P, dh=P, T=3, V=100, out=P, stream=NULL)
        a.update(kw)
        return L.fp8bs_logprobs_bwd(*a.values())

    for fn in (call, back):
        assert fn(T=0, x=NULL) == 0
        assert fn(dtype=2) == -4
        for kw in (dict(T=-1), dict(V=0), dict(stride=99)):
            assert fn(**kw) == -2, kw
        for kw in (dict(V=(1 << 20) + 1, stride=1 << 21), dict(T=1 << 31), dict(T=1 << 24), dict(stride=1 << 31)):
            assert fn(**kw) == -7, kw
        assert fn(x=MIS) == -3 and fn(x=P + 1, dtype=1) == -3
    for top in (-1, 101, 65):
        assert call(top=top) == -2
    for name in ("x", "y", "lp", "h", "norm", "rank", "ti", "tl", "ws"):
        assert call(**{name: NULL}) == -1, name
    for name in ("y", "lp", "h", "norm", "rank", "ti", "tl", "ws"):
        assert call(**{name: MIS}) == -3, name
    for name in ("x", "y", "norm", "h", "dl", "dh", "out"):
        assert back(**{name: NULL}) == -1, name
        assert back(**{name: MIS}) == -3, name
    ws = L.fp8bs_logprobs_workspace_bytes
    assert ws(3, 100, 5) > 0 and ws(3, 100, 65) == -2 and ws(-1, 100, 0) == -2 and ws(1, 1 << 21, 0) == -7


def test_binding_refusals():
    import torch
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    cu = torch.tensor([0, 4], dtype=i32)
    lat, rope = torch.zeros(4, 512, dtype=bf), torch.zeros(4, 64, dtype=bf)
    cache = torch.zeros(3, 16, 256, dtype=u8), torch.zeros(3, 16, 16, dtype=u8), torch.zeros(3, 16, 64, dtype=bf)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_mla_cache_write(lat, rope, cache, cu[None, :1], cu[:1], cu)
    with pytest.raises(ValueError, match="latent must be"):
        fb.fp8bs_mla_cache_write(lat[:, :100], rope, cache, cu[None, :1], cu[:1], cu)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_mla_cache_read(cache, cu[None, :1], cu[:1], cu, 4)
    with pytest.raises(TypeError, match="torch tensor"):
        fb.fp8bs_mla_cache_read([], cu[None, :1], cu[:1], cu, 4)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_mla_decode_fp4(torch.zeros(1, 1, 4, 576, dtype=bf), cache, cu[None], cu[:1], 0.1)
    with pytest.raises(ValueError, match="q must be"):
        fb.fp8bs_mla_decode_fp4_shared(lat, cache, cu, cu[:1], cu[None], cu[:1], 0.1)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_moe_tokens(lat, cu[None], cu[None].float(), lat, lat, lat, lat)
    with pytest.raises(ValueError, match="on a GPU"):
        fb.fp8bs_logprobs(lat, cu)
    with pytest.raises(ValueError, match="logits must be"):
        fb.fp8bs_logprobs_bwd(lat[0], cu, lat, lat, lat, lat)
