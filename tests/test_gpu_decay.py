"""Linear attention with a decay for each head on the GPU against its 64-bit
form: prompt, gradient and single tokens."""

import math

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu

G = [0.0, float("-inf"), -1e-4, -0.05, -3.0]  # no decay, no memory, slow, usual, a few tokens


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def make(B, H, L, d, dtype, layout, seed=0, n=3):
    """n operands [B, H, L, d]: contiguous, inside one projection's output, or at odd addresses and strides (which TMA
    does not take)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)
    if layout == "packed":
        x = z(B, L, n, H, d)
        return [x[:, :, i].transpose(1, 2) for i in range(n)]
    if layout == "odd":
        x = z(B, H, L, n * (d + 1) + 1)
        return [x[..., i * (d + 1) + 1:i * (d + 1) + 1 + d] for i in range(n)]
    return [z(B, H, L, d) for _ in range(n)]


def log_decay(H):
    return torch.tensor([G[h % len(G)] for h in range(H)], dtype=torch.float32, device="cuda")


def on_tensor_cores(dtype, layout):
    return dtype == torch.bfloat16 and layout != "odd"


def within(x, value, bound, what):
    e = (x.cpu().double() - value).abs()
    worst = float((e / bound).max()) if e.numel() else 0.0
    assert worst <= 1.0, (what, worst, float(e.max()))


def check_prompt(nats, q, k, v, g, tc, lens=None, state=None, scale=0.0, **kw):
    B, H, L, d = q.shape
    out, last = nats.decay_attn(q, k, v, g, scale=scale, lens=lens, state=state, return_state=True, **kw)
    torch.cuda.synchronize()
    s = scale or 1 / math.sqrt(d)
    n = [L] * B if lens is None else lens.tolist()
    rows = ref.batch(lambda q, k, v, st, n: ref.attn(q, k, v, g.cpu(), s, n, st), q, k, v, state, lens=n, L=L)
    for b, (o, size, S, S_size) in enumerate(rows):
        within(out[b], o, ref.out_bound(o, size, d, L, q.dtype, tc), ("out", b))
        within(last[b], S, ref.state_bound(S_size, L, tc), ("state", b))
    return out, last


SIZES = [(1, 1, 1), (2, 5, 2), (1, 3, 31), (2, 2, 64), (1, 5, 65), (1, 2, 127), (2, 3, 128), (1, 5, 129), (1, 2, 255),
         (3, 5, 300), (1, 5, 1000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "packed", "odd"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_prompt(nats, size, layout, d, dtype):
    B, H, L = size
    q, k, v = make(B, H, L, d, dtype, layout)
    gen = torch.Generator(device="cuda").manual_seed(1)
    state = torch.randn(B, H, d, d, generator=gen, device="cuda") * 3 if L % 2 else None
    check_prompt(nats, q, k, v, log_decay(H), on_tensor_cores(dtype, layout), state=state)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "odd"])
def test_prompt_padded(nats, layout, d, dtype):
    """Lengths of every kind, also outside 0 .. L; what lies behind a sequence's end is NaN and infinite."""
    L = 400
    lens = torch.tensor([400, 0, 1, 127, 128, 129, 256, 399, 31], dtype=torch.int32, device="cuda")
    B, H = len(lens), 5
    q, k, v = make(B, H, L, d, dtype, layout)
    for x in (q, k, v):
        for b, n in enumerate(lens.tolist()):
            x[b, :, n:, ::2] = float("nan")
            x[b, :, n:, 1::2] = float("inf")
    state = torch.randn(B, H, d, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    out, last = check_prompt(nats, q, k, v, log_decay(H), on_tensor_cores(dtype, layout), lens=lens, state=state)
    for b, n in enumerate(lens.tolist()):
        assert (out[b, :, n:] == 0).all()
    assert torch.equal(last[1], state[1])
    far = lens.clone()
    far[0], far[1] = 1000, -7
    out2, last2 = nats.decay_attn(q, k, v, log_decay(H), lens=far, state=state, return_state=True)
    assert torch.equal(out, out2) and torch.equal(last, last2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_cut(nats, d, dtype):
    """Few heads and a long sequence: segments, with ends inside them and ahead of them."""
    B, H, L = 2, 1, 3333
    q, k, v = make(B, H, L, d, dtype, "packed")
    dims = nats._native.DecayDims(B, H, L, d, 0 if dtype == torch.bfloat16 else 1, 0.0)
    assert nats._native.lib.nats_decay_attn_workspace_size(dims) > 0
    state = torch.randn(B, H, d, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    for g in (0.0, -0.01, float("-inf")):
        gt = torch.full((1,), g, device="cuda")
        check_prompt(nats, q, k, v, gt, dtype == torch.bfloat16, state=state)
        check_prompt(nats, q, k, v, gt, dtype == torch.bfloat16, state=state,
                     lens=torch.tensor([3000, 70], dtype=torch.int32, device="cuda"))
        check_prompt(nats, q, k, v, gt, dtype == torch.bfloat16)


@pytest.mark.parametrize("L", [100, 3333])
def test_state_in_place(nats, L):
    q, k, v = make(2, 2, L, 64, torch.bfloat16, "heads")
    g = torch.tensor([-0.01, -0.2], device="cuda")
    s = torch.randn(2, 2, 64, 64, device="cuda")
    out, last = nats.decay_attn(q, k, v, g, state=s, return_state=True)
    mine = s.clone()
    out2, got = nats.decay_attn(q, k, v, g, state=mine, state_out=mine)
    assert got.data_ptr() == mine.data_ptr() and torch.equal(mine, last) and torch.equal(out, out2)


@pytest.mark.parametrize("L", [300, 2500])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_same_bits(nats, dtype, L):
    q, k, v, u = make(1, 3, L, 128, dtype, "heads", n=4)
    g = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    a = nats.decay_attn(q, k, v, g, return_state=True)
    b = nats.decay_attn(q, k, v, g, return_state=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    a, b = (nats.decay_attn_bwd(u, q, k, v, g, state_grad=True) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def check_grad(nats, u, q, k, v, g, tc, lens=None, state=None, dstate=None, scale=0.0, **kw):
    B, H, L, d = q.shape
    r = nats.decay_attn_bwd(u, q, k, v, g, scale=scale, lens=lens, state=state, dstate_out=dstate, state_grad=True, **kw)
    torch.cuda.synchronize()
    s = scale or 1 / math.sqrt(d)
    n = [L] * B if lens is None else lens.tolist()
    rows = ref.batch(lambda u, q, k, v, st, ds, n: ref.attn_bwd(u, q, k, v, g.cpu(), s, n, st, ds), u, q, k, v, state,
                     dstate, lens=n, L=L)
    for b, row in enumerate(rows):
        for name, (x, size) in zip(("dq", "dk", "dv"), row):
            within(r[name][b], x, ref.out_bound(x, size, d, L, q.dtype, tc), (name, b))
        within(r["dstate"][b], row[3][0], ref.state_bound(row[3][1], L, tc), ("dstate", b))
    return r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("size", [(1, 1, 1), (2, 5, 2), (1, 5, 33), (2, 3, 128), (1, 5, 129), (2, 5, 300), (1, 5, 1000)],
                         ids=str)
def test_gradient(nats, size, layout, d, dtype):
    B, H, L = size
    u, q, k, v = make(B, H, L, d, dtype, layout, n=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    st = [torch.randn(B, H, d, d, generator=gen, device="cuda") * 3 if L % 2 else None for _ in range(2)]
    check_grad(nats, u, q, k, v, log_decay(H), on_tensor_cores(dtype, layout), state=st[0], dstate=st[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("layout", ["heads", "odd"])
def test_gradient_padded(nats, layout, d, dtype):
    L = 300
    lens = torch.tensor([300, 0, 1, 127, 128, 129, 257], dtype=torch.int32, device="cuda")
    B, H = len(lens), 5
    u, q, k, v = make(B, H, L, d, dtype, layout, n=4)
    for x in (u, q, k, v):
        for b, n in enumerate(lens.tolist()):
            x[b, :, n:] = float("nan")
    gen = torch.Generator(device="cuda").manual_seed(2)
    st = [torch.randn(B, H, d, d, generator=gen, device="cuda") for _ in range(2)]
    r = check_grad(nats, u, q, k, v, log_decay(H), on_tensor_cores(dtype, layout), lens=lens, state=st[0], dstate=st[1])
    for b, n in enumerate(lens.tolist()):
        assert all((r[x][b, :, n:] == 0).all() for x in ("dq", "dk", "dv"))
    assert torch.equal(r["dstate"][1], st[1][1]) or (r["dstate"][1] - st[1][1]).abs().max() <= 2 * ref.U * st[1][1].abs().max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_gradient_cut(nats, d, dtype):
    B, H, L = 2, 1, 2999
    u, q, k, v = make(B, H, L, d, dtype, "heads", n=4)
    dims = nats._native.DecayDims(B, H, L, d, 0 if dtype == torch.bfloat16 else 1, 0.0)
    assert nats._native.lib.nats_decay_attn_bwd_workspace_size(dims) > 0
    gen = torch.Generator(device="cuda").manual_seed(4)
    st = [torch.randn(B, H, d, d, generator=gen, device="cuda") for _ in range(2)]
    for g in (0.0, -0.01):
        gt = torch.full((1,), g, device="cuda")
        check_grad(nats, u, q, k, v, gt, dtype == torch.bfloat16, state=st[0], dstate=st[1], scale=0.3)
        check_grad(nats, u, q, k, v, gt, dtype == torch.bfloat16, state=st[0], dstate=st[1],
                   lens=torch.tensor([2600, 64], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("size", [(1, 1), (3, 5), (40, 16)], ids=str)
def test_step(nats, size, odd, d, dtype):
    B, H = size
    q, k, v = (x[:, :, 0] for x in make(B, H, 1, d, dtype, "odd" if odd else "packed"))
    g = log_decay(H)
    s = torch.randn(B, H, d, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    mine = s.clone()
    out = nats.decay_attn_step(q, k, v, g, mine)
    torch.cuda.synchronize()
    rows = ref.batch(lambda q, k, v, st, n: ref.attn(q, k, v, g.cpu(), 1 / math.sqrt(d), 1, st), q[:, :, None], k[:, :, None],
                     v[:, :, None], s, lens=[1] * B, L=1)
    for b, (o, size, S, S_size) in enumerate(rows):
        within(out[b], o[:, 0], ref.out_bound(o, size, d, 1, dtype, False)[:, 0], b)
        within(mine[b], S, S_size * 4 * ref.U + 1e-37, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_prompt_then_tokens(nats, dtype):
    """A prompt's state carries single tokens on as the longer prompt would."""
    B, H, L, T, d = 2, 5, 150, 7, 128
    q, k, v = make(B, H, L + T, d, dtype, "packed")
    g = log_decay(H)
    _, state = nats.decay_attn(q[:, :, :L], k[:, :, :L], v[:, :, :L], g, return_state=True)
    outs = [nats.decay_attn_step(q[:, :, L + t], k[:, :, L + t], v[:, :, L + t], g, state) for t in range(T)]
    rows = ref.batch(lambda q, k, v, n: ref.attn(q, k, v, g.cpu(), 1 / math.sqrt(d), n, None), q, k, v, lens=[L + T] * B,
                     L=L + T)
    tc = dtype == torch.bfloat16
    for b, (o, size, S, S_size) in enumerate(rows):
        bound = ref.out_bound(o, size, d, L + T, dtype, False) + size * (2.0 ** -16 if tc else 0.0)
        within(torch.stack(outs, 2)[b], o[:, L:], bound[:, L:], b)
        within(state[b], S, ref.state_bound(S_size, L + T, tc), b)


def test_prompt_in_parts(nats):
    """A prompt in uneven parts through the state equals one call, but for the state's rounding on the way."""
    q, k, v = make(1, 5, 700, 64, torch.float32, "heads")
    g = log_decay(5)
    whole, last = nats.decay_attn(q, k, v, g, return_state=True)
    state, parts = None, []
    for a, b in ((0, 1), (1, 130), (130, 130), (130, 651), (651, 700)):
        o, state = nats.decay_attn(q[:, :, a:b], k[:, :, a:b], v[:, :, a:b], g, state=state, return_state=True)
        parts.append(o)
    rows = ref.batch(lambda q, k, v, n: ref.attn(q, k, v, g.cpu(), 1 / 8, n, None), q, k, v, lens=[700], L=700)
    o, size, S, S_size = rows[0]
    within(torch.cat(parts, 2)[0], o, ref.out_bound(o, size, 64, 700, torch.float32, False), "parts")
    within(whole[0], o, ref.out_bound(o, size, 64, 700, torch.float32, False), "whole")
    within(state[0], S, ref.state_bound(S_size, 700, False), "state")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_cut_padded_with_garbage(nats, d, dtype):
    """Segments whose chunks end inside a tile, NaN behind them, forward and backward; lengths at a segment's edges."""
    B, H, L = 5, 1, 2600
    u, q, k, v = make(B, H, L, d, dtype, "heads", n=4)
    lens = torch.tensor([2600, 2500, 1, 257, 1300], dtype=torch.int32, device="cuda")
    for x in (u, q, k, v):
        for b, n in enumerate(lens.tolist()):
            x[b, :, n:] = float("nan")
    gt = torch.full((1,), -0.01, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(6)
    st = [torch.randn(B, H, d, d, generator=gen, device="cuda") for _ in range(2)]
    tc = dtype == torch.bfloat16
    check_prompt(nats, q, k, v, gt, tc, lens=lens, state=st[0])
    check_grad(nats, u, q, k, v, gt, tc, lens=lens, state=st[0], dstate=st[1])
    nats.decay_attn_check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_shared_and_given(nats, dtype):
    """Keys and values that all heads share (expanded), outputs in given tensors of other layouts, and a call without
    a state, whose output is that of the call with one, but for the state's parts."""
    B, H, L, d = 2, 5, 333, 64
    q, k, v = make(B, H, L, d, dtype, "heads")
    k, v = k[:, :1].expand(B, H, L, d), v[:, :1].expand(B, H, L, d)
    g = log_decay(H)
    want, _ = check_prompt(nats, q, k, v, g, False)
    out = torch.full((B, L, 2, H, d), 7.0, dtype=dtype, device="cuda")
    assert nats.decay_attn(q, k, v, g, out=out[:, :, 1].transpose(1, 2)).data_ptr() == out[:, :, 1].data_ptr()
    assert torch.equal(out[:, :, 1].transpose(1, 2), want) and (out[:, :, 0] == 7).all()
    q, k, v, u = make(B, H, L, d, dtype, "heads", n=4)
    want = nats.decay_attn(q, k, v, g)
    nats.decay_attn(q, k, v, g, out=out[:, :, 1].transpose(1, 2))
    assert torch.equal(out[:, :, 1].transpose(1, 2), want) and (out[:, :, 0] == 7).all()
    grads = nats.decay_attn_bwd(u, q, k, v, g)
    buf = torch.full((B, L, 4, H, d), 7.0, dtype=dtype, device="cuda")
    views = {n: buf[:, :, i].transpose(1, 2) for i, n in enumerate(("dq", "dk", "dv"))}
    r = nats.decay_attn_bwd(u, q, k, v, g, **views)
    assert all(torch.equal(r[n], grads[n]) for n in grads) and (buf[:, :, 3] == 7).all()
    rows = ref.batch(lambda q, k, v, n: ref.attn(q, k, v, g.cpu(), d ** -0.5, n, None), q, k, v, lens=[L] * B, L=L)
    for b, (o, size, _, _) in enumerate(rows):
        within(want[b], o, ref.out_bound(o, size, d, L, dtype, dtype == torch.bfloat16) + size * 2.0 ** -16, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L", [200, 3333])
def test_no_state_out(nats, L, d, dtype):
    """Calls that give no state out, whole and cut into segments: decayed values as two bf16 numbers (2^-16)."""
    u, q, k, v = make(1, 2, L, d, dtype, "packed", n=4)
    g = torch.tensor([-0.002, -0.3], device="cuda")
    tc = dtype == torch.bfloat16
    out, r = nats.decay_attn(q, k, v, g), nats.decay_attn_bwd(u, q, k, v, g)
    assert set(r) == {"dq", "dk", "dv"}
    o, size, _, _ = ref.attn(q[0].cpu(), k[0].cpu(), v[0].cpu(), g.cpu(), d ** -0.5, L, None)
    within(out[0], o, ref.out_bound(o, size, d, L, dtype, tc) + size * (2.0 ** -16 if tc else 0.0), "out")
    grads = ref.attn_bwd(u[0].cpu(), q[0].cpu(), k[0].cpu(), v[0].cpu(), g.cpu(), d ** -0.5, L, None, None)
    for name, (x, size) in zip(("dq", "dk", "dv"), grads):
        within(r[name][0], x, ref.out_bound(x, size, d, L, dtype, tc) + size * (2.0 ** -16 if tc else 0.0), name)
    nats.decay_attn_check()


def test_two_streams(nats):
    """Two calls at once, each cut into segments with a workspace of its own."""
    a, b = (make(1, 1, 4000, 128, torch.bfloat16, "heads", seed=s) for s in (1, 2))
    g = torch.full((1,), -0.02, device="cuda")
    want = [nats.decay_attn(*x, g, return_state=True) for x in (a, b)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [nats.decay_attn(*x, g, return_state=True, stream=t) for x, t in zip((a, b), s)]
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_empty(nats):
    g = torch.zeros(3, device="cuda")
    for shape in ((0, 3, 5, 64), (2, 3, 0, 64)):
        x = torch.randn(*shape, device="cuda")
        s = torch.randn(shape[0], 3, 64, 64, device="cuda")
        out, last = nats.decay_attn(x, x, x, g, state=s, return_state=True)
        assert out.shape == x.shape and torch.equal(last, s)
        r = nats.decay_attn_bwd(x, x, x, x, g, dstate_out=s, state_grad=True)
        assert r["dq"].shape == x.shape and torch.equal(r["dstate"], s)
        assert (nats.decay_attn(x, x, x, g, return_state=True)[1] == 0).all()
    x = torch.randn(2, 0, 64, device="cuda")
    assert nats.decay_attn_step(x, x, x, torch.zeros(0, device="cuda"), torch.zeros(2, 0, 64, 64, device="cuda")).shape == x.shape


def test_captured(nats):
    """Captured once, replayed on new contents, on another stream."""
    q, k, v, u = make(2, 2, 300, 128, torch.bfloat16, "heads", n=4)
    g = torch.tensor([-0.01, -0.2], device="cuda")
    s = torch.zeros(2, 2, 128, 128, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        nats.decay_attn(q, k, v, g, state=s, return_state=True)
        nats.decay_attn_bwd(u, q, k, v, g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, last = nats.decay_attn(q, k, v, g, state=s, return_state=True)
        r = nats.decay_attn_bwd(u, q, k, v, g, dstate_out=last)
        o1 = nats.decay_attn_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, last)
    for seed in (7, 8):
        for x, y in zip((q, k, v, u), make(2, 2, 300, 128, torch.bfloat16, "heads", seed=seed, n=4)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        out2, last2 = nats.decay_attn(q, k, v, g, state=s, return_state=True)
        r2 = nats.decay_attn_bwd(u, q, k, v, g, dstate_out=last2)
        o2 = nats.decay_attn_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], g, last2)
        assert torch.equal(out, out2) and torch.equal(last, last2) and torch.equal(o1, o2)
        assert all(torch.equal(r[n], r2[n]) for n in r)


def test_other_stream(nats):
    """On a stream given, with outputs read on the current one and inputs freed before the call has run."""
    side = torch.cuda.Stream()
    q, k, v = make(2, 4, 2000, 128, torch.bfloat16, "heads")
    g = torch.full((4,), -0.05, device="cuda")
    want = nats.decay_attn(q, k, v, g)
    torch.cuda.synchronize()
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    side.wait_stream(torch.cuda.current_stream())
    out = nats.decay_attn(q2, k2, v2, g, stream=side)
    del q2, k2, v2
    torch.full((3 * q.numel(),), float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)


def test_refusals(nats):
    x = torch.randn(2, 3, 8, 64, device="cuda")
    g = torch.zeros(3, device="cuda")
    s = torch.zeros(2, 3, 64, 64, device="cuda")
    bad = [
        (ValueError, lambda: nats.decay_attn(x, x[:, :2], x, g)),
        (TypeError, lambda: nats.decay_attn(x, x.bfloat16(), x, g)),
        (TypeError, lambda: nats.decay_attn(x.half(), x.half(), x.half(), g)),
        (ValueError, lambda: nats.decay_attn(x.cpu(), x, x, g)),
        (ValueError, lambda: nats.decay_attn(x[0], x[0], x[0], g)),
        (ValueError, lambda: nats.decay_attn(x.mT, x.mT, x.mT, g)),
        (ValueError, lambda: nats.decay_attn(x, x, x, g[:2])),
        (TypeError, lambda: nats.decay_attn(x, x, x, g.double())),
        (TypeError, lambda: nats.decay_attn(x, x, x, None)),
        (TypeError, lambda: nats.decay_attn(x, x, x, g, lens=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: nats.decay_attn(x, x, x, g, lens=torch.zeros(3, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: nats.decay_attn(x, x, x, g, state=s[:1])),
        (TypeError, lambda: nats.decay_attn(x, x, x, g, state=s.bfloat16())),
        (ValueError, lambda: nats.decay_attn(x, x, x, g, state=s.mT)),
        (ValueError, lambda: nats.decay_attn(x, x, x, g, out=x[:1, :, :, :].expand(2, 3, 8, 64))),
        (ValueError, lambda: nats.decay_attn(x, x, x, g, scale=1e-300)),
        (nats.NatsError, lambda: nats.decay_attn(x, x, x, g, scale=-1.0)),
        (nats.NatsError, lambda: nats.decay_attn(x, x, x, g, scale=1e-39)),
        (nats.NatsError, lambda: nats.decay_attn(x[..., :32], x[..., :32], x[..., :32], g)),
        (ValueError, lambda: nats.decay_attn_bwd(x[:1], x, x, x, g)),
        (ValueError, lambda: nats.decay_attn_bwd(x, x, x, x, g, dstate_out=s[:1])),
        (TypeError, lambda: nats.decay_attn_bwd(x, x, x, x, g, dq=x.bfloat16())),
        (TypeError, lambda: nats.decay_attn_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, None)),
        (ValueError, lambda: nats.decay_attn_step(x, x, x, g, s)),
        (ValueError, lambda: nats.decay_attn_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, s.mT)),
        (ValueError, lambda: nats.decay_attn_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], g, s,
                                                  out=x[:1, :, 0].expand(2, 3, 64))),
    ]
    for i, (e, f) in enumerate(bad):
        with pytest.raises(e):
            f()
            pytest.fail(f"case {i}")
