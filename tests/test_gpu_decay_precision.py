"""The precision of linear attention with a decay as it shows in the mean: the
worst-case bounds of the other tests leave room for a state summed from values of
16 bits, these do not.

States that are given out (tensor cores): a decayed value is three bf16 numbers,
its fp32 value, so products are exact.  A chunk's sum is 8 steps of 16 products,
each cut off at 2 U of the sum so far (U = 2^-24), U each on average and 8 U in
all if the sum were whole from the first; the three parts' sums, the carry and
the factor of a chunk round, U each, at random.  Below 16.8 U = 1e-6.  Two parts
leave half a step of half a step out, 2^-16 of each value at most; in the mean, what
the first part leaves being anywhere in its half step and its own binade setting the
second one's, 2^-16 / sqrt(21) / 1.5 = 2.2e-6.

fp32 outputs: two factors of 2^-23 at most and a product of 2^-22 left out, less
than half of that in the mean (below 4 U), sums as above without the cuts.

bf16 outputs: three roundings, of the scores, the state and the result, each half
a step (2^-8) over sqrt(3) and 0.7: 1.6e-3 each, 2.8e-3 together."""

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def off(x, want):
    """rms(error) / rms(value)."""
    x, want = x.cpu().double(), want.double()
    return float((x - want).square().mean().sqrt() / want.square().mean().sqrt())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [64, 500, 3333])  # whole, whole, cut into segments
def test_precision(nats, L, d, dtype):
    gen = torch.Generator(device="cuda").manual_seed(L + d)
    H = 2
    u, q, k, v = (torch.randn(1, H, L, d, generator=gen, device="cuda").to(dtype) for _ in range(4))
    s, ds = (torch.randn(1, H, d, d, generator=gen, device="cuda") for _ in range(2))
    g = torch.tensor([-0.003, -0.05], device="cuda")
    out, last = nats.decay_attn(q, k, v, g, state=s, return_state=True)
    r = nats.decay_attn_bwd(u, q, k, v, g, state=s, dstate_out=ds, state_grad=True)
    c = [x[0].cpu() for x in (u, q, k, v)]
    o, _, S, _ = ref.attn(*c[1:], g.cpu(), d ** -0.5, L, s[0].cpu())
    grads = [x for x, _ in ref.attn_bwd(*c, g.cpu(), d ** -0.5, L, s[0].cpu(), ds[0].cpu())]
    outputs = 1e-6 if dtype == torch.float32 else 2.8e-3
    assert off(last[0], S) < 1e-6 and off(r["dstate"][0], grads[3]) < 1e-6
    assert off(out[0], o) < outputs
    for name, want in zip(("dq", "dk", "dv"), grads):
        assert off(r[name][0], want) < outputs, name
    if dtype == torch.bfloat16:
        # without a state given out: decayed values of two parts, seen only through products in bf16
        assert off(nats.decay_attn(q, k, v, g, state=s)[0], o) < outputs
        r = nats.decay_attn_bwd(u, q, k, v, g, state=s, dstate_out=ds)
        assert all(off(r[n][0], want) < outputs for n, want in zip(("dq", "dk", "dv"), grads))
