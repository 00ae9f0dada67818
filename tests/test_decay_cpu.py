"""Host side of layer norm and of linear attention with a decay: refusals
through the C ABI before any launch, and the 64-bit gradients against
differences."""

import pytest
import torch

import decay_ref as ref

A = 0x10000000  # a fake but aligned address: validation rejects before touching it


@pytest.fixture(scope="module")
def nat():
    from linear_attention_nats_gb300 import build as b

    b.build()
    from linear_attention_nats_gb300 import _native

    return _native


def _decay(nat, what, **kw):
    d = dict(B=1, H=2, L=9000, d=64, dtype=0, scale=0.0)
    p = dict(q=A, k=A, v=A, g=A, lens=None, s=None, out=A, so=None, ws=A, nws=1 << 40, u=A, dso=None, dq=A, dk=A, dv=A, dsi=None,
             st=True)
    for n, v in kw.items():
        (d if n in d else p)[n] = v
    dm = nat.DecayDims(*[d[n] for n in ("B", "H", "L", "d", "dtype", "scale")])
    s = nat.Strides(1 << 20, 1 << 14, 64) if p["st"] else None
    if what == "fwd":
        return nat.lib.nats_decay_attn(dm, p["q"], s, p["k"], s, p["v"], s, p["g"], p["lens"], p["s"], p["out"], s, p["so"],
                                       p["ws"], p["nws"], None)
    if what == "bwd":
        return nat.lib.nats_decay_attn_bwd(dm, p["u"], s, p["q"], s, p["k"], s, p["v"], s, p["g"], p["lens"], p["s"], p["dso"],
                                           p["dq"], s, p["dk"], s, p["dv"], s, p["dsi"], p["ws"], p["nws"], None)
    return nat.lib.nats_decay_attn_step(dm, p["q"], s, p["k"], s, p["v"], s, p["g"], p["s"], p["out"], s, None)


COMMON = [(dict(B=-1), 2), (dict(H=-1), 2), (dict(L=-1), 2), (dict(d=96), 6), (dict(d=256), 6), (dict(dtype=2), 3),
          (dict(scale=-1.0), 9), (dict(scale=float("inf")), 9), (dict(scale=float("nan")), 9), (dict(scale=1e-39), 9),
          (dict(B=1 << 20, H=8), 6), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1),
          (dict(st=False), 1), (dict(q=A + 1), 4), (dict(v=A + 2, dtype=1), 4), (dict(g=A + 2), 4), (dict(B=0), 0),
          (dict(H=0), 0)]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(L=(1 << 30) + 1), 6), (dict(out=None), 1), (dict(ws=None), 1),
                                              (dict(ws=A + 8), 4), (dict(nws=16), 5), (dict(lens=A + 2), 4), (dict(s=A + 2), 4),
                                              (dict(so=A + 1), 4), (dict(L=0), 0)])
def test_prompt_refusals(nat, kw, code):
    assert _decay(nat, "fwd", **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(L=(1 << 30) + 1), 6), (dict(u=None), 1), (dict(dq=None), 1), (dict(dk=None), 1),
                                              (dict(dv=None), 1), (dict(ws=None), 1), (dict(ws=A + 8), 4), (dict(nws=16), 5),
                                              (dict(dso=A, dsi=A), 9), (dict(dso=A + 2), 4), (dict(L=0), 0)])
def test_gradient_refusals(nat, kw, code):
    assert _decay(nat, "bwd", **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(L=2), 2), (dict(L=0), 2), (dict(out=None), 1), (dict(s=None), 1),
                                              (dict(s=A + 4), 4)])
def test_step_refusals(nat, kw, code):
    assert _decay(nat, "step", **{**dict(L=1, s=A), **kw}) == code


def test_decay_workspace(nat):
    f, g = nat.lib.nats_decay_attn_workspace_size, nat.lib.nats_decay_attn_bwd_workspace_size
    assert f(nat.DecayDims(1, 1, 100, 96, 0, 0.0)) == 0 and f(nat.DecayDims(4, 64, 8192, 128, 0, 0.0)) == 0
    assert f(nat.DecayDims(1, 1, 0, 64, 0, 0.0)) == 0 and f(nat.DecayDims(1, 1, 16, 64, 0, 0.0)) == 0
    assert f(nat.DecayDims(1, 1, 65536, 128, 0, 0.0)) >= 2 * 128 * 128 * 4
    assert g(nat.DecayDims(1, 1, 65536, 128, 0, 0.0)) >= 4 * 128 * 128 * 4
    assert f(nat.DecayDims(1, 1, 1 << 30, 128, 0, 0.0)) <= 64 * 128 * 128 * 4


def _norm(nat, bwd, **kw):
    d = dict(B=1, H=1, L=4, D=64, dtype=0, eps=1e-6)
    p = dict(x=A, w=A, b=A, out=A, u=A, dw=A, db=A, ws=A, nws=1 << 30, st=True)
    for n, v in kw.items():
        (d if n in d else p)[n] = v
    dm = nat.NormDims(*[d[n] for n in ("B", "H", "L", "D", "dtype", "eps")])
    s = nat.Strides(1 << 20, 1 << 14, 64) if p["st"] else None
    if bwd:
        return nat.lib.nats_layer_norm_bwd(dm, p["u"], s, p["x"], s, p["w"], p["out"], s, p["dw"], p["db"], p["ws"], p["nws"], None)
    return nat.lib.nats_layer_norm(dm, p["x"], s, p["w"], p["b"], p["out"], s, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 2), (dict(H=-1), 2), (dict(L=-1), 2), (dict(D=0), 2), (dict(D=16385), 6), (dict(B=1 << 16, L=1 << 15), 6),
    (dict(dtype=2), 3), (dict(eps=-1e-3), 9), (dict(eps=float("nan")), 9), (dict(x=None), 1), (dict(out=None), 1),
    (dict(st=False), 1), (dict(x=A + 1), 4), (dict(out=A + 2, dtype=1), 4), (dict(w=A + 2), 4)])
def test_norm_refusals(nat, bwd, kw, code):
    assert _norm(nat, bwd, **kw) == code


def test_norm_sum_refusals(nat):
    assert _norm(nat, True, u=None) == 1 and _norm(nat, True, ws=None) == 1 and _norm(nat, True, ws=A + 8) == 4
    assert _norm(nat, True, dw=A + 2) == 4 and _norm(nat, True, nws=4 * 2 * 64 * 4 - 1) == 5
    assert nat.lib.nats_layer_norm_bwd_workspace_size(nat.NormDims(1, 1, 4, 64, 0, 1e-6)) == 4 * 2 * 64 * 4
    assert nat.lib.nats_layer_norm_bwd_workspace_size(nat.NormDims(1, 1, 4, 0, 0, 1e-6)) == 0
    assert _norm(nat, False, B=0) == 0 and _norm(nat, False, L=0) == 0


def _differences(f, x, u, h=1e-4):
    """<u, f(x + h e)> - <u, f(x - h e)> over 2 h for every entry e."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view(x.shape)
        g.view(-1)[i] = (u * (f(x + e) - f(x - e))).sum() / (2 * h)
    return g


def test_norm_gradient_form():
    gen = torch.Generator().manual_seed(0)
    x, u = torch.randn(3, 11, dtype=torch.float64, generator=gen), torch.randn(3, 11, dtype=torch.float64, generator=gen)
    w, b = torch.randn(11, dtype=torch.float64, generator=gen), torch.randn(11, dtype=torch.float64, generator=gen)
    dx, dw, db = ref.norm_bwd(u, x, w, 0.1)
    for got, want in ((dx, _differences(lambda x: ref.norm(x, w, b, 0.1), x, u)),
                      (dw, _differences(lambda w: ref.norm(x, w, b, 0.1), w, u)),
                      (db, _differences(lambda b: ref.norm(x, w, b, 0.1), b, u))):
        assert (got - want).abs().max() < 1e-6


@pytest.mark.parametrize("n", [0, 1, 4, 5])
def test_attn_gradient_form(n):
    """The output's and the last state's gradients together, with tokens behind the sequence's end."""
    gen = torch.Generator().manual_seed(1)
    z = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)
    q, k, v, u, S, R = z(2, 5, 3), z(2, 5, 3), z(2, 5, 3), z(2, 5, 3), z(2, 3, 3), z(2, 3, 3)
    g = torch.tensor([-0.3, 0.0], dtype=torch.float64)

    def f(q=q, k=k, v=v, S=S):
        o, _, last, _ = ref.attn(q, k, v, g, 0.7, n, S)
        return torch.cat([o.reshape(-1), last.reshape(-1)])

    both = torch.cat([u.reshape(-1), R.reshape(-1)])
    got = [x for x, _ in ref.attn_bwd(u, q, k, v, g, 0.7, n, S, R)]
    want = [_differences(lambda x: f(**{name: x}), t, both) for name, t in (("q", q), ("k", k), ("v", v), ("S", S))]
    for x, y in zip(got, want):
        assert (x - y).abs().max() < 1e-6


def test_attn_recurrence():
    """The matrix form against the recurrence, token by token."""
    gen = torch.Generator().manual_seed(2)
    z = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)
    q, k, v, S = z(3, 9, 4), z(3, 9, 4), z(3, 9, 4), z(3, 4, 4)
    g = torch.tensor([-0.2, 0.0, float("-inf")], dtype=torch.float64)
    o, _, last, _ = ref.attn(q, k, v, g, 0.5, 7, S)
    for t in range(7):
        S = torch.exp(g)[:, None, None] * S + v[:, t, :, None] * k[:, t, None, :]
        assert (o[:, t] - 0.5 * (S @ q[:, t, :, None])[..., 0]).abs().max() < 1e-12
    assert (last - S).abs().max() < 1e-12 and (o[:, 7:] == 0).all()


@pytest.mark.parametrize("back", [False, True])
def test_decay_table(back):
    """The tensor-core kernel's table of decays: four copies shifted by an entry each, read four entries at a time from a
    16-byte boundary, give every row its decays to the columns of a block, and stay inside their copy."""
    copy, g = 168, -0.1
    tab = [0.0] * (4 * copy)
    for e in range(4 * copy):
        y = e % copy + e // copy
        m = y - 31 if back else 127 - y
        tab[e] = g * m if m >= 0 else None
    for i in range(128):
        at = (31 if back else 127) - i
        w = i // 32
        for blk in (range(w, 4) if back else range(w + 1)):
            for j in range(0, 32, 4):
                a = (at & 3) * copy + (at & ~3) + 32 * blk + j
                assert a % 4 == 0 and (at & 3) * copy <= a and a + 3 < (at & 3) * copy + 160
                for e in range(4):
                    m = 32 * blk + j + e - i if back else i - 32 * blk - j - e
                    assert tab[a + e] == (g * m if m >= 0 else None)


@pytest.mark.parametrize("L", [1, 64, 127, 128, 129, 1000, 70000])
@pytest.mark.parametrize("segs", [1, 2, 7])
@pytest.mark.parametrize("C", [64, 128])
def test_segments_cover(L, segs, C):
    """Segments of whole chunks cover the tokens once, in both directions, whatever the length."""
    chunks = -(-L // C)
    per = -(-chunks // segs)
    if -(-chunks // per) != segs:
        return
    for n in {0, 1, C - 1, C, L // 2, L}:
        if n > L:
            continue
        seen = 0
        for seg in range(segs):
            t0, t1 = seg * per * C, min(seg * per * C + per * C, L)
            m = max(0, min(t1, n) - t0)
            N = -(-m // C)
            assert t0 == seen or m == 0
            for back in (False, True):
                part_c, part_n = (0 if back else N - 1), m - (N - 1) * C
                tokens = [part_n if c == part_c else C for c in range(N)]
                assert sum(tokens) == m and all(0 < t <= C for t in tokens)
            seen += m
        assert seen == n
