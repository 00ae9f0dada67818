"""Query / key norm and rotation and its gradient against plain 64-bit forms."""

from fractions import Fraction

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def nats():
    from linear_attention_nats_gb300 import build

    build.build()
    import linear_attention_nats_gb300 as n

    return n


def _operand(rng, B, H, L, d, dtype, layout):
    """[B, H, L, d] on the CPU: contiguous, inside a wider [B, L, W] buffer, or at odd offsets and strides."""
    if layout == "contiguous":
        return torch.randn(B, H, L, d, generator=rng).to(dtype)
    pad = 2 * d if layout == "fused" else 3
    off = d if layout == "fused" else 1
    buf = torch.randn(B, L, H * d + pad, generator=rng).to(dtype)
    return buf[..., off:off + H * d].unflatten(-1, (H, d)).transpose(1, 2)


def _dev(t):
    """The same tensor on the GPU with the same offset and strides."""
    if t is None:
        return None
    s = torch.empty(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype).set_(t.untyped_storage()).cuda()
    return s.as_strided(t.shape, t.stride(), t.storage_offset())


CASES = [
    # B, L, Hq, Hk, d, rot, interleaved, dtype, norm, layout, weights
    (1, 1, 1, 1, 64, 64, False, BF, True, "contiguous", True),
    (1, 1, 16, 16, 128, 128, False, BF, True, "fused", True),
    (2, 3, 5, 1, 128, 128, True, BF, True, "fused", True),
    (3, 67, 12, 4, 64, 32, True, F32, True, "contiguous", True),
    (2, 130, 4, 2, 128, 112, False, F32, True, "fused", True),
    (2, 33, 3, 3, 64, 8, False, BF, True, "odd", True),
    (1, 65, 2, 1, 128, 48, True, F32, True, "odd", True),
    (2, 9, 7, 2, 64, 0, False, BF, True, "contiguous", True),
    (2, 9, 7, 2, 128, 128, False, BF, False, "fused", False),
    (1, 257, 8, 8, 128, 128, False, F32, True, "fused", False),
    (1, 40, 0, 3, 64, 64, False, BF, True, "contiguous", True),
    (1, 40, 3, 0, 64, 64, True, F32, True, "contiguous", True),
    (5, 2049, 3, 1, 64, 64, False, BF, True, "fused", True),
]


def _make(case, seed, far=100000):
    B, L, Hq, Hk, d, rot, inter, dtype, norm, layout, weights = case
    rng = torch.Generator().manual_seed(seed)
    q, k = _operand(rng, B, Hq, L, d, dtype, layout), _operand(rng, B, Hk, L, d, dtype, layout)
    wq = 1 + 0.3 * torch.randn(d, generator=rng) if weights else None
    wk = 1 + 0.3 * torch.randn(d, generator=rng) if weights else None
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64) if rot else None
    pos = torch.randint(0, far, (B, L), generator=rng)
    return q, k, wq, wk, f, pos


@pytest.mark.parametrize("case", CASES)
def test_forward(nats, case):
    B, L, Hq, Hk, d, rot, inter, dtype, norm, layout, weights = case
    q, k, wq, wk, f, pos = _make(case, 11)
    oq, ok = nats.qk_norm_rope(_dev(q), _dev(k), _dev(wq), _dev(wk), _dev(f), _dev(pos), interleaved=inter, norm=norm)
    assert oq.is_contiguous() and ok.is_contiguous()
    for x, w, o in ((q, wq, oq), (k, wk, ok)):
        y = ref.norm_rotate(x, w, pos, f, inter, norm, 1e-6)
        z = ref.norm_rotate(x, w, pos, None, inter, norm, 1e-6)
        assert ((o.cpu().double() - y).abs() <= ref.rope_bound(y, z, rot, inter, dtype)).all()


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("grad,dx", [("x", "x"), ("f32", "x"), ("f32", "f32"), ("x", "f32")])
def test_backward(nats, case, grad, dx):
    B, L, Hq, Hk, d, rot, inter, dtype, norm, layout, weights = case
    q, k, wq, wk, f, pos = _make(case, 12)
    gt, xt = F32 if grad == "f32" else dtype, F32 if dx == "f32" else dtype
    rng = torch.Generator().manual_seed(5)
    gq, gk = _operand(rng, B, Hq, L, d, gt, layout), _operand(rng, B, Hk, L, d, gt, "contiguous")
    out = {n: torch.full_like(_dev(x), 7.0, dtype=xt) for n, x in (("dq", q), ("dk", k))}
    r = nats.qk_norm_rope_bwd(_dev(gq), _dev(gk), _dev(q), _dev(k), _dev(wq), _dev(wk), _dev(f), _dev(pos),
                              interleaved=inter, norm=norm, **out)
    assert r["dq"] is out["dq"] and ("dw_q" in r) == norm
    for n, g, x, w in (("q", gq, q, wq), ("k", gk, k, wk)):
        e, dw, pair = ref.norm_rotate_bwd(g, x, w, pos, f, inter, norm, 1e-6)
        b = ref.rope_bwd_bound(g, x, w, pos, f, inter, norm, 1e-6, e, xt)
        assert ((r["d" + n].cpu().double() - e).abs() <= b).all()
        if not norm:
            continue
        if rot:  # the magnitudes of a turned entry's terms: |u| is at most its pair's sum of |dy|
            i, j = ref.pairs_of(rot, inter)
            u = g.double().abs()
            s = u[..., i] + u[..., j]
            u = u.clone()
            u[..., i], u[..., j] = s, s.clone()
            pair = (u * x.double().abs() / (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()).sum((0, 1, 2))
        # a term to 30 U of those, summed at most 200 steps deep (a lane's rows, the warp, the CTA, the CTAs)
        assert ((r["dw_" + n].cpu().double() - dw).abs() <= 256 * ref.U * pair + 1e-30).all()


# more tokens than warps run at once, few rows each: a group of lanes takes a token of its own
MANY = [
    (3, 1307, 2, 1, 128, 128, False, BF, True, "fused", True),
    (1, 3931, 1, 1, 128, 48, True, F32, True, "contiguous", True),
    (2, 2001, 4, 2, 64, 32, True, BF, True, "fused", False),
    (7, 701, 0, 3, 64, 64, False, F32, True, "contiguous", True),
    (1, 4099, 13, 0, 128, 112, False, BF, False, "fused", False),
]


@pytest.mark.parametrize("case", MANY)
def test_forward_of_many_tokens(nats, case):
    test_forward(nats, case)


@pytest.mark.parametrize("case", MANY)
@pytest.mark.parametrize("grad,dx", [("x", "x"), ("f32", "x")])
def test_backward_of_many_tokens(nats, case, grad, dx):
    test_backward(nats, case, grad, dx)


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 128)])
def test_many_tokens_in_place_and_in_parts(nats, dtype, d):
    """The same bits in place, and from calls of so few tokens that the rows of one lie side by side."""
    rng = torch.Generator().manual_seed(23)
    q, k = torch.randn(1, 3, 4099, d, generator=rng).to(dtype).cuda(), torch.randn(1, 1, 4099, d, generator=rng).to(dtype).cuda()
    g = [torch.randn(x.shape, generator=rng).to(dtype).cuda() for x in (q, k)]
    f = nats.rope_inv_freq(d)
    y = nats.qk_norm_rope(q, k, None, None, f, pos0=7)
    r = nats.qk_norm_rope_bwd(*g, q, k, None, None, f, pos0=7)
    for a in range(0, 4099, 1000):
        part = [x[:, :, a:a + 1000] for x in (q, k, *g)]
        for whole, p in zip(y, nats.qk_norm_rope(*part[:2], None, None, f, pos0=7 + a)):
            assert torch.equal(whole[:, :, a:a + 1000], p)
        rp = nats.qk_norm_rope_bwd(*part[2:], *part[:2], None, None, f, pos0=7 + a)
        assert torch.equal(r["dq"][:, :, a:a + 1000], rp["dq"]) and torch.equal(r["dk"][:, :, a:a + 1000], rp["dk"])
    gi = [x.clone() for x in g]
    ri = nats.qk_norm_rope_bwd(*gi, q, k, None, None, f, pos0=7, dq=gi[0], dk=gi[1])
    for n in ("dq", "dk", "dw_q", "dw_k"):
        assert torch.equal(ri[n], r[n])
    yi = nats.qk_norm_rope(q, k, None, None, f, pos0=7, out_q=q, out_k=k)
    assert torch.equal(yi[0], y[0]) and torch.equal(yi[1], y[1])


def test_backward_against_differences(nats):
    """<dx, v> = d/dt <dy, y(x + t v)> by central differences of the 64-bit
    forward; h = 1e-5 leaves h^2 of third derivatives, about 1e-9, and the
    fp32 gradient its rounding, 40 U of the magnitudes."""
    case = (2, 19, 4, 2, 64, 48, False, F32, True, "contiguous", True)
    q, k, wq, wk, f, pos = _make(case, 21, far=4096)
    rng = torch.Generator().manual_seed(6)
    gq, gk = torch.randn(q.shape, generator=rng), torch.randn(k.shape, generator=rng)
    r = nats.qk_norm_rope_bwd(gq.cuda(), gk.cuda(), q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), f.cuda(), pos.cuda())
    h = 1e-5
    for n, g, x, w in (("q", gq, q, wq), ("k", gk, k, wk)):
        fwd = lambda xx, ww: (g.double() * ref.norm_rotate(xx, ww, pos, f, False, True, 1e-6)).sum()
        v, vw = torch.randn(x.shape, generator=rng).double(), torch.randn(64, generator=rng).double()
        num = (fwd(x.double() + h * v, w) - fwd(x.double() - h * v, w)) / (2 * h)
        got = (r["d" + n].cpu().double() * v).sum()
        scale = (r["d" + n].cpu().double() * v).abs().sum()
        assert abs(num - got) <= 1e-6 * scale
        num = (fwd(x, w.double() + h * vw) - fwd(x, w.double() - h * vw)) / (2 * h)
        got = (r["dw_" + n].cpu().double() * vw).sum()
        assert abs(num - got) <= 1e-5 * (r["dw_" + n].cpu().double() * vw).abs().sum()


def test_far_positions(nats):
    """Angles at positions up to 2^40, the exact turn taken in rational
    arithmetic from the frequency's own bits and 60 digits of pi."""
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    pos = torch.tensor([[0, 1, 12345, 1 << 20, (1 << 31) + 7, (1 << 40) + 3, -5, -(1 << 33)]])
    f = torch.tensor([0.9999, 1.0, 0.31, 1e-3, 3.7e-6, 2.5, 1e-12, 0.0], dtype=torch.float64)
    x = torch.zeros(1, 1, 8, 64)
    x[..., :8] = 1.0
    y, _ = nats.qk_norm_rope(x.cuda(), x.cuda(), None, None, f.cuda(), pos.cuda(), norm=False)
    import math

    for t, p in enumerate(pos[0].tolist()):
        for i, w in enumerate(f.tolist()):
            turn = Fraction(w) * p / two_pi
            turn -= turn.numerator // turn.denominator
            a = 2 * math.pi * float(turn)
            # phase: |p| (2^-62.5 of the frequency and one unit) 2^-64 turns, 2^-32 cut off, then 6 U
            tol = 2 * math.pi * (abs(p) * (w / 6.28 * 2 ** -62.5 + 2 ** -64) + 2 ** -32) + 6 * ref.U
            assert abs(float(y[0, 0, t, i]) - math.cos(a)) <= tol
            assert abs(float(y[0, 0, t, 8 + i]) - math.sin(a)) <= tol


def test_positions_default_shared_and_offset(nats):
    rng = torch.Generator().manual_seed(3)
    q, k = torch.randn(2, 3, 17, 64, generator=rng).cuda(), torch.randn(2, 1, 17, 64, generator=rng).cuda()
    f = nats.rope_inv_freq(64)
    a = nats.qk_norm_rope(q, k, None, None, f, pos0=1000)
    b = nats.qk_norm_rope(q, k, None, None, f, torch.arange(1000, 1017, device="cuda"))
    c = nats.qk_norm_rope(q, k, None, None, f, torch.arange(1000, 1017, device="cuda").expand(2, 17))
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_in_place_and_into_strided_outputs(nats):
    rng = torch.Generator().manual_seed(4)
    qkv = torch.randn(2, 21, 9 * 128, generator=rng).to(BF).cuda()
    parts = lambda t: (t[..., :4 * 128].unflatten(-1, (4, 128)).transpose(1, 2),
                       t[..., 4 * 128:6 * 128].unflatten(-1, (2, 128)).transpose(1, 2))
    f = nats.rope_inv_freq(128)
    want = nats.qk_norm_rope(*parts(qkv), None, None, f)
    rest = qkv[..., 6 * 128:].clone()
    q, k = parts(qkv)
    nats.qk_norm_rope(q, k, None, None, f, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[..., 6 * 128:], rest)


def test_zero_extents(nats):
    f = nats.rope_inv_freq(64)
    z = lambda *s: torch.zeros(s, device="cuda")
    for B, L in ((0, 4), (2, 0)):
        q, k = z(B, 3, L, 64), z(B, 1, L, 64)
        oq, ok = nats.qk_norm_rope(q, k, None, None, f)
        assert oq.shape == q.shape
        r = nats.qk_norm_rope_bwd(oq, ok, q, k, None, None, f)
        assert (r["dw_q"] == 0).all() and (r["dw_k"] == 0).all()


def test_backward_repeats_bit_for_bit(nats):
    case = (4, 513, 12, 4, 128, 128, False, BF, True, "fused", True)
    q, k, wq, wk, f, pos = (_dev(x) for x in _make(case, 31))
    gq, gk = torch.randn_like(q, dtype=F32), torch.randn_like(k, dtype=F32)
    a = nats.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, f, pos)
    b = nats.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, f, pos)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_other_stream_and_graph(nats):
    case = (2, 65, 4, 2, 64, 64, False, BF, True, "contiguous", True)
    q, k, wq, wk, f, pos = (_dev(x) for x in _make(case, 41))
    want = nats.qk_norm_rope(q, k, wq, wk, f, pos)
    grad = nats.qk_norm_rope_bwd(*want, q, k, wq, wk, f, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nats.qk_norm_rope(q, k, wq, wk, f, pos, stream=s)
    back = nats.qk_norm_rope_bwd(*want, q, k, wq, wk, f, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(back[n], grad[n]) for n in grad)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = nats.qk_norm_rope(q, k, wq, wk, f, pos)
        b = nats.qk_norm_rope_bwd(*o, q, k, wq, wk, f, pos)
    q.mul_(-0.5)
    g.replay()
    want = nats.qk_norm_rope(q, k, wq, wk, f, pos)
    grad = nats.qk_norm_rope_bwd(*want, q, k, wq, wk, f, pos)
    assert all(torch.equal(x, y) for x, y in zip(o, want)) and all(torch.equal(b[n], grad[n]) for n in grad)


def test_offsets_beyond_32_bits(nats):
    """Rows 2^20 entries apart: the last tokens lie behind the 2^31st entry."""
    T, S = 2200, 1 << 20
    buf = torch.empty(T * S, dtype=BF, device="cuda")
    q = buf.as_strided((1, 3, T, 64), (0, 128, S, 1))
    k = buf.as_strided((1, 2, T, 64), (0, 128, S, 1), 512)
    rng = torch.Generator().manual_seed(9)
    q0, k0 = torch.randn(1, 3, T, 64, generator=rng).to(BF), torch.randn(1, 2, T, 64, generator=rng).to(BF)
    q.copy_(q0), k.copy_(k0)
    f = nats.rope_inv_freq(64)
    want = nats.qk_norm_rope(q0.cuda(), k0.cuda(), None, None, f, pos0=5)
    grad = nats.qk_norm_rope_bwd(*want, q0.cuda(), k0.cuda(), None, None, f, pos0=5)
    got = nats.qk_norm_rope_bwd(*want, q, k, None, None, f, pos0=5)
    assert all(torch.equal(got[n], grad[n]) for n in grad)
    nats.qk_norm_rope(q, k, None, None, f, pos0=5, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_refusals(nats):
    x = torch.zeros(1, 2, 4, 64, device="cuda")
    f = nats.rope_inv_freq(64)
    with pytest.raises(TypeError):
        nats.qk_norm_rope(x.half(), x.half(), None, None, f)
    with pytest.raises(TypeError):
        nats.qk_norm_rope(x, x.bfloat16(), None, None, f)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x.cpu(), x, None, None, f)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x, x[:, :, :3], None, None, f)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x.transpose(2, 3), x.transpose(2, 3), None, None, f)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x, x, None, None, f, out_q=x[:, :1].expand(1, 2, 4, 64))
    with pytest.raises(TypeError):
        nats.qk_norm_rope(x, x, None, None, f.float())
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x, x, torch.ones(63, device="cuda"), None, f)
    with pytest.raises(nats.NatsError):
        nats.qk_norm_rope(x, x, None, None, nats.rope_inv_freq(12))  # not a multiple of 8
    with pytest.raises(nats.NatsError):
        nats.qk_norm_rope(x, x, None, None, nats.rope_inv_freq(72))  # beyond d
    with pytest.raises(nats.NatsError):
        nats.qk_norm_rope(x, x, None, None, f, eps=-1.0)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x, x, None, None, f, pos0=1 << 63)
    with pytest.raises(ValueError):
        nats.qk_norm_rope(x, x, None, None, f, torch.zeros(2, 4, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        nats.qk_norm_rope(x, x, None, None, f, torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(nats.NatsError):
        nats.qk_norm_rope_bwd(x.bfloat16(), x.bfloat16(), x, x, None, None, f)  # fp32 inputs, bf16 gradients


def test_feeds_the_hybrid_layer(nats):
    """q, k from one projection, keys brought to unit length by the weight d^(-1/2), then the layer: the same as the
    layer on queries and keys prepared in 64 bits and rounded, to the rounding of its inputs (half a bf16 step moves
    the output by at most a few of its own; the layer's bar is 1e-2 of the largest entry)."""
    B, H, L, d = 1, 2, 256, 64
    rng = torch.Generator().manual_seed(8)
    qkv = torch.randn(B, L, 3, H, d, generator=rng).to(BF)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    f, pos = torch.tensor([10000.0 ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64), torch.arange(L).expand(B, L)
    wk = torch.full((d,), d ** -0.5)
    dq = qkv.cuda()
    q2, k2 = nats.qk_norm_rope(dq[:, :, 0].transpose(1, 2), dq[:, :, 1].transpose(1, 2), None, wk.cuda(), f.cuda())
    assert ((k2.float().norm(dim=-1) - 1).abs() < 2 ** -7).all()
    g, beta = -0.1 * torch.rand(B, H, L, generator=rng), torch.rand(B, H, L, generator=rng)
    sel = torch.randint(0, 2, (B, H, L // 64), generator=rng).to(torch.uint8).cuda()
    w_g = 0.02 * torch.randn(H, d, generator=rng)
    run = lambda a, b: nats.hybrid_fwd(a, b, v.contiguous().cuda(), g.cuda(), beta.cuda(), None, None, w_g.cuda(),
                                       sel_in=sel).float()
    got = run(q2, k2)
    want = run(ref.norm_rotate(q, None, pos, f, False, True, 1e-6).to(BF).contiguous().cuda(),
               ref.norm_rotate(k, wk, pos, f, False, True, 1e-6).to(BF).contiguous().cuda())
    assert (got - want).abs().max() <= 1e-2 * want.abs().max()
