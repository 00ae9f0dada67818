"""Layer norm's arithmetic where a mean's rounding shows: rows of one value, and
rows far from zero beside their spread."""

import math

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
# one piece, groups within a warp, of two warps and of a CTA; whole pieces, pairs and entry by entry
DS = [64, 65, 100, 128, 1000, 1001, 1002, 1024, 2048, 4096, 4100, 8192, 16384]


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


@TYPES
@pytest.mark.parametrize("D", DS)
@pytest.mark.parametrize("N", [3, 20000])  # (more rows than the short rows' kernel starts from)
def test_rows_of_one_value(nats, N, D, dtype):
    """z is 0: the output is the bias, the weights' gradient 0, whatever the value."""
    if N * D > 1 << 26:
        N = 1300
    value = torch.tensor([3.3, 100.1, 1000.1, -9999.9, 1e5 / 3, 1e-3, 1.7e18], device="cuda")
    x = value.repeat(-(-N // 7))[:N, None].expand(N, D).to(dtype).contiguous()
    gen = torch.Generator(device="cuda").manual_seed(0)
    w, b = (torch.randn(D, generator=gen, device="cuda") for _ in range(2))
    u = torch.randn(N, D, generator=gen, device="cuda").to(dtype)
    assert torch.equal(nats.layer_norm(x, w, b), b.to(dtype).expand(N, D))
    assert (nats.layer_norm(x) == 0).all()
    r = nats.layer_norm_bwd(u, x, w)
    assert (r["dw"] == 0).all() and torch.isfinite(r["dx"]).all()


@pytest.mark.parametrize("D", DS)
@pytest.mark.parametrize("mean", [1e3, 3e4, -1e6])
@pytest.mark.parametrize("spread", [1.0, 1e-2])
def test_far_rows(nats, spread, mean, D):
    """The mean that is subtracted is off by its own rounding, U |mean|, and by depth U of the spread and of what the
    first sum was off by (depth U |mean|); so is x - mean.  The variance takes no part of it, the sums of distances and
    squares are depth U off each: with n = sqrt(var + eps), |z| is off by (U |mean| (1 + depth^2 U) + depth U spread) / n
    + |z| (depth + 10) U."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(50, D, generator=gen, device="cuda") * spread + mean
    y = nats.layer_norm(x)
    xd = x.double()
    mu, var = xd.mean(-1, keepdim=True), xd.var(-1, keepdim=True, unbiased=False)
    n, depth = (var + 1e-6).sqrt(), 2 * math.log2(D + 1) + 40
    z = (xd - mu) / n
    bound = (ref.U * mu.abs() * (1 + depth ** 2 * ref.U) + depth * ref.U * var.sqrt()) / n + z.abs() * (depth + 10) * ref.U
    # (what the first mean was off by, squared, is taken out of the variance: depth U of it and of itself remain)
    first = (depth * ref.U * mu.abs()) ** 2 / n ** 2
    bound = bound + z.abs() * first * 4 * depth * ref.U + 1e-37
    assert ((y.double() - z).abs() <= bound).all(), float(((y.double() - z).abs() / bound).max())
