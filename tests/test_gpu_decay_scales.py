"""Linear attention with a decay at scales far from the usual ones: the states'
gradients go in and out as they are, whatever the scale."""

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def within(x, value, bound, what):
    e = (x.cpu().double() - value).abs()
    assert bool((e <= bound).all()), (what, float((e / bound).max()), float(e.max()))


def operands(L, d, dtype, std, H=3):
    gen = torch.Generator(device="cuda").manual_seed(3)
    u, q, k, v = ((torch.randn(1, H, L, d, generator=gen, device="cuda") * std).to(dtype) for _ in range(4))
    st = [torch.randn(1, H, d, d, generator=gen, device="cuda") for _ in range(2)]
    return u, q, k, v, torch.tensor([-0.02, 0.0, -1.5], device="cuda")[:H].contiguous(), st


# the operands' size keeps the definition's own values inside fp32: scale times an entry and a product of two of them
@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [200, 2600])
@pytest.mark.parametrize("scale,std", [(1e-37, 1.0), (1e-20, 1.0), (1e20, 1.0), (1e37, 1e-3)])
def test_scales(nats, scale, std, L, d, dtype):
    u, q, k, v, g, (s, ds) = operands(L, d, dtype, std)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    # the least gradient of a state that a small scale's quotient would have taken out of range
    ds = ds * (100.0 if scale < 1 else 1.0)
    tc = dtype == torch.bfloat16
    out, last = nats.decay_attn(q, k, v, g, scale=scale, state=s, return_state=True)
    r = nats.decay_attn_bwd(u, q, k, v, g, scale=scale, state=s, dstate_out=ds, state_grad=True)
    c = lambda x: x[0].cpu()
    o, size, S, S_size = ref.attn(c(q), c(k), c(v), g.cpu(), scale, L, c(s))
    within(out[0], o, ref.out_bound(o, size, d, L, dtype, tc), "out")
    within(last[0], S, ref.state_bound(S_size, L, False), "state")
    rows = ref.attn_bwd(c(u), c(q), c(k), c(v), g.cpu(), scale, L, c(s), c(ds))
    for name, (x, size) in zip(("dq", "dk", "dv"), rows):
        within(r[name][0], x, ref.out_bound(x, size, d, L, dtype, tc), name)
    within(r["dstate"][0], rows[3][0], ref.state_bound(rows[3][1], L, False), "dstate")


@TYPES
@pytest.mark.parametrize("scale", [1e-37, 1e37])
def test_state_alone(nats, scale, dtype):
    """Without a gradient of the outputs, dstate is the decayed gradient of the last state: every digit of it."""
    u, q, k, v, g, (s, ds) = operands(300, 64, dtype, 1e-3)
    ds = ds * 1e-3
    r = nats.decay_attn_bwd(torch.zeros_like(u), q, k, v, g, scale=scale, state=s, dstate_out=ds, state_grad=True)
    want = torch.exp(g.double() * 300)[:, None, None] * ds[0].double()
    # 300 tokens in at most five chunks: a carry is off by 2 U, its factor by (g 300 + 2) U
    bound = want.abs() * (5 * 2 + 1.5 * 300 + 2) * ref.U + 1e-44
    within(r["dstate"][0], want.cpu(), bound.cpu(), "dstate")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = nats.decay_attn_bwd(u, q, k, v, g, scale=scale, lens=lens, dstate_out=ds, state_grad=True)
    assert torch.equal(r["dstate"], ds)  # an empty sequence's passes through
