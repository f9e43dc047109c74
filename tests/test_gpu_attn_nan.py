"""NaN in the attention operators on the GPU: a query that holds or sees one
says so, in out and in lse; it does not look like a query that sees no key. The
other queries' results keep their bits."""

import pytest
import torch

import fp8_block_scaled_x1_amd as fb

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
NAN = float("nan")


def _randn(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("Lq,Lk,H", [(40, 40, 2), (300, 300, 2), (40, 3000, 2), (300, 600, 200)],
                         ids=["one tile", "tiles", "in parts", "256-query blocks"])
def test_expanded(dev, Lq, Lk, H):
    g = torch.Generator().manual_seed(1)
    q, kv, kr = (_randn(g, *s).to(dev) for s in ((Lq, H, 192), (Lk, H, 256), (Lk, 64)))
    dout = _randn(g, Lq, H, 128).to(dev)
    cq, ck = (torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (Lq, Lk))
    out, lse = fb.fp8bs_mla_prefill(q, kv, kr, cq, ck, SCALE)
    bad = q.clone()
    bad[17, 1, 100] = NAN                       # one query of one head
    o2, l2 = fb.fp8bs_mla_prefill(bad, kv, kr, cq, ck, SCALE)
    assert torch.all(torch.isnan(o2[17, 1])) and torch.isnan(l2[1, 17])
    o2[17, 1], l2[1, 17] = out[17, 1], lse[1, 17]
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # the rotary key of token Lk - 5: the last five queries see it, in every head
    badr = kr.clone()
    badr[Lk - 5, 3] = NAN
    o3, l3 = fb.fp8bs_mla_prefill(q, kv, badr, cq, ck, SCALE)
    assert torch.all(torch.isnan(o3[-5:])) and torch.all(torch.isnan(l3[:, -5:]))
    assert torch.equal(o3[:-5], out[:-5]) and torch.equal(l3[:, :-5], lse[:, :-5])
    # and a gradient of theirs is not a number either
    dq, dkv, dk_rope = fb.fp8bs_mla_prefill_bwd(dout, q, kv, badr, o3, l3, cq, ck, SCALE)
    assert torch.all(torch.isnan(dq[-5:])) and torch.all(torch.isnan(dkv[Lk - 5])) and torch.all(torch.isnan(dk_rope[Lk - 5]))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,prefix", [(50, 0), (700, 0), (300, 200)], ids=["whole", "joined", "behind a prefix"])
def test_absorbed(dev, kind, n, prefix):
    g = torch.Generator().manual_seed(2)
    page, B, H = 16, 3, 4
    per, npre = -(-n // page), -(-prefix // page)
    x = _randn(g, B * per + npre, page, 576).to(dev)
    cache = x
    if kind == "fp8":
        codes, scales = fb.fp8_quant_act_1x128(x[..., :512].reshape(-1, 512).contiguous())
        cache = (codes.reshape(*x.shape[:2], 512), scales.t().reshape(*x.shape[:2], 4).contiguous(), x[..., 512:].contiguous())
    table = (npre + torch.arange(B * per, dtype=torch.int32).reshape(B, per)).to(dev)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev)
    pt, pl = torch.arange(npre, dtype=torch.int32, device=dev), torch.tensor([prefix], dtype=torch.int32, device=dev)
    q = _randn(g, B, 1, H, 576).to(dev)

    def call(q):
        if prefix:
            return fb.fp8bs_mla_decode_shared(q, cache, pt, pl, table, lens, SCALE)
        return fb.fp8bs_mla_decode(q, cache, table, lens, SCALE)

    out, lse = call(q)
    assert torch.all(torch.isfinite(out)) and torch.all(torch.isfinite(lse))
    bad = q.clone()
    bad[1, 0, 2, 40] = NAN
    o2, l2 = call(bad)
    assert torch.all(torch.isnan(o2[1, 0, 2])) and torch.isnan(l2[1, 0, 2])
    o2[1, 0, 2], l2[1, 0, 2] = out[1, 0, 2], lse[1, 0, 2]
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # a rotary number of request 2's token n - 3 (not a value): all of its queries, nobody else's
    (cache if kind == "bf16" else cache[2])[npre + 2 * per + (n - 3) // page, (n - 3) % page, -7] = NAN
    o3, l3 = call(q)
    assert torch.all(torch.isnan(o3[2])) and torch.all(torch.isnan(l3[2]))
    assert torch.equal(o3[:2], out[:2]) and torch.equal(l3[:2], lse[:2])
