"""Norm + rotation with frequencies that are not finite."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nats():
    from linear_attention_nats_gb300 import build

    build.build()
    import linear_attention_nats_gb300 as n

    return n


@pytest.mark.parametrize("tokens,Hq,Hk", [(9, 12, 4), (5000, 1, 1)])  # a token's rows side by side; a token each
@pytest.mark.parametrize("d,dtype,inter", [(64, F32, False), (64, BF, True), (128, BF, False), (128, F32, True)])
def test_frequencies_that_are_not_finite(nats, tokens, Hq, Hk, d, dtype, inter):
    """Their pairs have no angle: cos(p inf) is NaN, also at position 0.  The other entries are what they are without."""
    rng = torch.Generator().manual_seed(d)
    q, k = (torch.randn(1, h, tokens, d, generator=rng).to(dtype).cuda() for h in (Hq, Hk))
    rot = d - 16
    f = nats.rope_inv_freq(rot)
    pos = torch.arange(tokens, device="cuda")
    pairs = [0, 3, 4, 11, rot // 2 - 1]
    values = [math.inf, math.nan, -math.inf, -math.nan, math.inf]
    ends = [e for i in pairs for e in ((2 * i, 2 * i + 1) if inter else (i, i + rot // 2))]
    bad = f.clone()
    bad[pairs] = torch.tensor(values, dtype=torch.float64, device="cuda")
    others = [e for e in range(d) if e not in ends]
    good, got = (nats.qk_norm_rope(q, k, None, None, x, pos, interleaved=inter) for x in (f, bad))
    for a, b in zip(good, got):
        assert torch.isnan(b[..., ends]).all() and torch.equal(a[..., others], b[..., others])
    # the gradient: of the rotation alone those entries, under the norm whole rows (each entry has a part of the others)
    a, b = (nats.qk_norm_rope_bwd(q, k, q, k, None, None, x, pos, interleaved=inter, norm=False) for x in (f, bad))
    for n in ("dq", "dk"):
        assert torch.isnan(b[n][..., ends]).all() and torch.equal(a[n][..., others], b[n][..., others])
    a, b = (nats.qk_norm_rope_bwd(q, k, q, k, None, None, x, pos, interleaved=inter) for x in (f, bad))
    for n in ("q", "k"):
        assert torch.isnan(b["d" + n]).all()
        assert torch.isnan(b["dw_" + n][ends]).all() and torch.equal(a["dw_" + n][others], b["dw_" + n][others])
    # into a cache
    pages = -(-tokens // 16)
    c = nats.PagedCache.empty(pages, 16, Hk, d, 1, pages, dtype=dtype)
    c.table.copy_(torch.arange(pages, dtype=torch.int32)[None])
    oq = nats.paged_append(c, k, k, q=q, norm=True, inv_freq=bad, interleaved=inter)
    kept = c.k_pages.transpose(1, 2).reshape(-1, Hk, d)[:tokens].transpose(0, 1)
    for a, b in zip(good, (oq, kept[None])):
        assert torch.isnan(b[..., ends]).all() and torch.equal(a[..., others], b[..., others])
