"""Layer norm and its gradient on the GPU against their 64-bit forms."""

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu

TYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def rows(shape, dtype, seed=0, mean=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return (z(*shape) * z(*shape[:-1], 1).exp() + mean * z(*shape[:-1], 1)).to(dtype)


def weights(D, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(D, generator=gen, device="cuda"), torch.randn(D, generator=gen, device="cuda")


def within(x, value, bound, what=""):
    e = (x.cpu().double() - value).abs()
    worst = float((e / bound).max()) if e.numel() else 0.0
    assert worst <= 1.0, (what, worst, float(e.max()))


def check(nats, x, u, w, b, eps=1e-6):
    D = x.shape[-1]
    y = nats.layer_norm(x, w, b, eps=eps)
    r = nats.layer_norm_bwd(u, x, w, eps=eps)
    torch.cuda.synchronize()
    c = lambda t: None if t is None else t.cpu()
    assert y.shape == x.shape and y.is_contiguous() and r["dx"].shape == x.shape
    within(y, ref.norm(c(x), c(w), c(b), eps), ref.norm_bound(c(x), c(w), c(b), eps, x.dtype), "y")
    want, bounds = ref.norm_bwd(c(u), c(x), c(w), eps), ref.norm_bwd_bound(c(u), c(x), c(w), eps, x.dtype)
    within(r["dx"].reshape(-1, D), want[0], bounds[0], "dx")
    within(r["dw"], want[1], bounds[1], "dw")
    within(r["db"], want[2], bounds[2], "db")


# lengths of rows at the edges of each way a row is held, whole pieces and entry by entry
DS = [1, 2, 7, 31, 33, 64, 65, 66, 128, 256, 257, 258, 512, 777, 1000, 1024, 1025, 2048, 2049, 2050, 4096, 4098, 4104, 5000, 8192,
      8194, 8200, 16382, 16383, 16384]


@TYPES
@pytest.mark.parametrize("D", DS)
@pytest.mark.parametrize("N", [1, 37])
def test_rows(nats, N, D, dtype):
    check(nats, rows((N, D), dtype), rows((N, D), dtype, 2, 0.0), *weights(D))


@TYPES
@pytest.mark.parametrize("shape", [(5000, 64), (3000, 128), (700, 2048), (2500, 100), (160003, 64), (80001, 120), (40009, 256),
                                   (900, 1030)], ids=str)
def test_many_rows(nats, shape, dtype):
    check(nats, rows(shape, dtype), rows(shape, dtype, 2, 0.0), *weights(shape[-1]))


@TYPES
def test_no_weights(nats, dtype):
    x, u = rows((9, 192), dtype), rows((9, 192), dtype, 2, 0.0)
    check(nats, x, u, None, None)
    check(nats, x, u, weights(192)[0], None, eps=0.1)
    r = nats.layer_norm_bwd(u, x, weight_grads=False)
    assert set(r) == {"dx"} and torch.equal(r["dx"], nats.layer_norm_bwd(u, x)["dx"])


@TYPES
@pytest.mark.parametrize("d", [64, 128, 33])
def test_layouts(nats, d, dtype):
    """Heads inside [B, L, H, d], rows with gaps and odd addresses, an expanded input: the values of the plain layout."""
    x, u = rows((2, 7, 5, d), dtype).transpose(1, 2), rows((2, 7, 5, d), dtype, 2, 0.0).transpose(1, 2)
    w, b = weights(d)
    check(nats, x, u, w, b)
    want, g = nats.layer_norm(x.contiguous(), w, b), nats.layer_norm_bwd(u.contiguous(), x.contiguous(), w)
    assert torch.equal(nats.layer_norm(x, w, b), want)
    wide = rows((2, 5, 7, d + 3), dtype)
    wide[..., 1:1 + d] = x
    odd = wide[..., 1:1 + d]
    check(nats, odd, u, w, b)
    out = torch.empty((2, 7, 5, d), dtype=dtype, device="cuda").transpose(1, 2)
    assert nats.layer_norm(x, w, b, out=out) is out and torch.equal(out, want)
    dx = torch.empty((2, 5, 7, 2 * d), dtype=dtype, device="cuda")[..., :d]
    assert torch.equal(nats.layer_norm_bwd(u, x, w, dx=dx)["dx"], g["dx"])
    one = x[:, :1].expand(2, 5, 7, d)
    assert torch.equal(nats.layer_norm(one, w, b), want[:, :1].expand(2, 5, 7, d))
    deep = rows((2, 3, 4, 5, d), dtype)  # neighbours that follow one another are one
    assert torch.equal(nats.layer_norm(deep, w, b), nats.layer_norm(deep.reshape(-1, d), w, b).view(deep.shape))


@TYPES
def test_in_place(nats, dtype):
    w, b = weights(300)
    x, u = rows((1500, 300), dtype), rows((1500, 300), dtype, 2, 0.0)
    want, g = nats.layer_norm(x, w, b), nats.layer_norm_bwd(u, x, w)
    for mine in (u.clone(), None):
        y = x.clone()
        r = nats.layer_norm_bwd(mine if mine is not None else u, y, w, dx=mine if mine is not None else y)
        assert all(torch.equal(r[n], g[n]) for n in g)
    y = x.clone()
    assert torch.equal(nats.layer_norm(y, w, b, out=y), want)


@TYPES
def test_values(nats, dtype):
    """A constant row, a row far from zero, large and small rows; a NaN or an infinity stays in its own row."""
    x = rows((8, 96), dtype)
    x[1] = 3.0
    x[2] = 1000.0 + torch.arange(96, device="cuda") % 8 * 4
    x[3] *= 1e15
    x[4] *= 1e-12
    w, b = weights(96)
    check(nats, x, rows((8, 96), dtype, 2, 0.0), w, b)
    y = nats.layer_norm(x, w, b)
    x[5, 7], x[6, 0] = float("nan"), float("inf")
    z = nats.layer_norm(x, w, b)
    assert torch.isnan(z[5]).all() and torch.isnan(z[6]).all()
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(z[keep], y[keep])
    r = nats.layer_norm_bwd(torch.ones_like(x), x, w)
    assert torch.isfinite(r["dx"][keep]).all()


def test_many_entries(nats):
    """Rows behind the 2^31st entry."""
    N, D = (1 << 31) // 2048 + 1000, 2048
    x = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rows((3, D), torch.bfloat16)
    w, b = weights(D)
    y = nats.layer_norm(x, w, b, out=x)
    want = nats.layer_norm(rows((3, D), torch.bfloat16), w, b)
    assert torch.equal(y[-3:], want)


def test_empty_and_same_bits(nats):
    w, b = weights(64)
    x = torch.empty((0, 64), device="cuda")
    assert nats.layer_norm(x, w, b).shape == (0, 64)
    r = nats.layer_norm_bwd(x, x, w)
    assert (r["dw"] == 0).all() and (r["db"] == 0).all() and r["dx"].shape == (0, 64)
    assert nats.layer_norm(torch.empty((4, 0, 2, 64), device="cuda").transpose(0, 2)).shape == (2, 0, 4, 64)
    x, u = rows((4099, 64), torch.bfloat16), rows((4099, 64), torch.bfloat16, 2)
    a, c = nats.layer_norm_bwd(u, x, w), nats.layer_norm_bwd(u, x, w)
    assert all(torch.equal(a[n], c[n]) for n in a)
    one = rows((64,), torch.float32)
    assert torch.equal(nats.layer_norm(one, w, b), nats.layer_norm(one[None], w, b)[0])


def test_captured(nats):
    w, b = weights(256)
    x, u = rows((100, 256), torch.bfloat16), rows((100, 256), torch.bfloat16, 2)
    nats.layer_norm_bwd(u, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nats.layer_norm(x, w, b)
        r = nats.layer_norm_bwd(u, x, w)
    x.copy_(rows((100, 256), torch.bfloat16, 9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, nats.layer_norm(x, w, b))
    r2 = nats.layer_norm_bwd(u, x, w)
    assert all(torch.equal(r[n], r2[n]) for n in r)


def test_refusals(nats):
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    bad = [
        (TypeError, lambda: nats.layer_norm(x.half())),
        (TypeError, lambda: nats.layer_norm(None)),
        (ValueError, lambda: nats.layer_norm(x.cpu())),
        (ValueError, lambda: nats.layer_norm(x.t())),
        (ValueError, lambda: nats.layer_norm(x.sum())),
        (ValueError, lambda: nats.layer_norm(x, w[:32])),
        (TypeError, lambda: nats.layer_norm(x, w.bfloat16())),
        (ValueError, lambda: nats.layer_norm(x, torch.ones(128, device="cuda")[::2])),
        (TypeError, lambda: nats.layer_norm(x, out=x.bfloat16())),
        (ValueError, lambda: nats.layer_norm(x, out=x[:2])),
        (ValueError, lambda: nats.layer_norm(x, out=x[:1].expand(4, 64))),
        (nats.NatsError, lambda: nats.layer_norm(x, eps=-1.0)),
        (nats.NatsError, lambda: nats.layer_norm(x, eps=float("nan"))),
        (nats.NatsError, lambda: nats.layer_norm(torch.empty((2, 16385), device="cuda"))),
        (nats.NatsError, lambda: nats.layer_norm(torch.empty((2, 0), device="cuda"))),
        (ValueError, lambda: nats.layer_norm(torch.empty((2, 3, 4, 5, 64), device="cuda").permute(3, 1, 0, 2, 4))),
        (ValueError, lambda: nats.layer_norm_bwd(x[:2], x)),
        (TypeError, lambda: nats.layer_norm_bwd(x.bfloat16(), x)),
        (nats.NatsError, lambda: nats.layer_norm_bwd(x, x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (e, f) in enumerate(bad):
        with pytest.raises(e):
            f()
            pytest.fail(f"case {i}")
