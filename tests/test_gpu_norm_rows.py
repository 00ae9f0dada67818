"""Layer norm with many long rows, where a group of threads takes two of them
(forward) or goes through several (gradient): every row against its 64-bit form,
with an odd number of rows, rows that do not fill their pieces, in place and as
heads."""

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def inputs(N, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    z = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = (z(N, D) * z(N, 1).exp() + 2 * z(N, 1)).to(dtype)
    return x, z(N, D).to(dtype), 1 + 0.3 * z(D), z(D)


def within(x, value, bound, what):
    e = (x.double() - value).abs()
    assert bool((e <= bound).all()), (what, float((e / bound).max()))


# more than 1216 rows: two bf16 ones to a group from 512 entries on
@TYPES
@pytest.mark.parametrize("N", [1217, 1999])
@pytest.mark.parametrize("D", [512, 520, 1000, 1024, 1030, 2040, 2048, 4096, 4104, 8200, 16384])
def test_forward(nats, D, N, dtype):
    x, _, w, b = inputs(N, D, dtype)
    y = nats.layer_norm(x, w, b)
    within(y, ref.norm(x, w, b, 1e-6), ref.norm_bound(x, w, b, 1e-6, dtype), "y")
    mine = x.clone()
    assert torch.equal(nats.layer_norm(mine, w, b, out=mine), y)
    # rows at strides: with a gap behind each, inside [B, L, H, D]
    wide = torch.full((N, D + 8), float("nan"), dtype=dtype, device="cuda")
    wide[:, :D] = x
    assert torch.equal(nats.layer_norm(wide[:, :D], w, b), y)
    B, H, L = 1, 7, N // 7
    heads = x[:B * H * L].view(B, L, H, D).transpose(1, 2)
    out = torch.full((B, L, H, D), 7.0, dtype=dtype, device="cuda")
    nats.layer_norm(heads, w, b, out=out.transpose(1, 2))
    assert torch.equal(out.view(-1, D), y[:B * H * L])


# more rows than three to each group that the GPU holds, so that the copies ahead go round
@TYPES
@pytest.mark.parametrize("N,D", [(20001, 64), (16001, 256), (9001, 1000), (4801, 2040), (4801, 2048), (2401, 4096), (1301, 4104),
                                 (1301, 8192), (701, 8200), (701, 12288), (701, 16384), (4801, 1030), (1301, 4097)])
def test_gradient(nats, N, D, dtype):
    x, u, w, _ = inputs(N, D, dtype)
    r = nats.layer_norm_bwd(u, x, w)
    want, bounds = ref.norm_bwd(u, x, w, 1e-6), ref.norm_bwd_bound(u, x, w, 1e-6, dtype)
    for name, v, e in zip(("dx", "dw", "db"), want, bounds):
        within(r[name], v, e, name)
    for given in (u.clone(), x.clone()):
        is_u = torch.equal(given, u)
        mine = nats.layer_norm_bwd(given if is_u else u, x if is_u else given, w, dx=given)
        assert all(torch.equal(mine[n], r[n]) for n in r)
    H, L = 3, N // 3
    a, c = (t[:H * L].view(1, L, H, D).transpose(1, 2) for t in (u, x))
    mine, plain = nats.layer_norm_bwd(a, c, w), nats.layer_norm_bwd(u[:H * L], x[:H * L], w)
    assert torch.equal(mine["dx"].transpose(1, 2).reshape(-1, D), plain["dx"])
    within(mine["dw"], plain["dw"].double(), 2 * ref.norm_bwd_bound(u[:H * L], x[:H * L], w, 1e-6, dtype)[1], "dw of heads")
