"""Host side of the norm / rotation and paged-cache operators: refusals
through the C ABI before any launch, the fixed-point frequency and the deal of
tiles to CTAs as index models, and the 64-bit forms against each other."""

import ctypes
import math
import random
from fractions import Fraction

import pytest
import torch

import serving_ref as ref

A = 0x10000000  # a fake but aligned address: validation rejects before touching it


@pytest.fixture(scope="module")
def nat():
    from linear_attention_nats_gb300 import build as b

    b.build()
    from linear_attention_nats_gb300 import _native

    return _native


def _rope(nat, **kw):
    d = dict(B=1, L=4, Hq=2, Hk=1, d=64, rot=64, interleaved=0, norm=1, dtype=0, eps=1e-6)
    ptr = dict(q=A, k=A + 4096, f=A + 8192, oq=A + 16384, ok=A + 32768, wq=None, pos=None)
    for n, v in kw.items():
        (d if n in d else ptr)[n] = v
    dm = nat.RopeDims(*[d[n] for n in ("B", "L", "Hq", "Hk", "d", "rot", "interleaved", "norm", "dtype", "eps")])
    s = nat.Strides(512, 256, 64)
    return nat.lib.nats_qk_norm_rope(dm, ptr["q"], s, ptr["k"], s, ptr["wq"], None, ptr["f"], ptr["pos"], 0, 0,
                                     ptr["oq"], s, ptr["ok"], s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), 2), (dict(L=-1), 2), (dict(Hq=-2), 2), (dict(rot=12), 2), (dict(rot=72), 2), (dict(rot=-8), 2),
    (dict(d=96), 6), (dict(d=256), 6), (dict(dtype=5), 3), (dict(eps=-1.0), 9), (dict(eps=float("inf")), 9),
    (dict(q=None), 1), (dict(k=None), 1), (dict(f=None), 1), (dict(oq=None), 1), (dict(ok=None), 1),
    (dict(q=A + 1), 4), (dict(wq=A + 2), 4), (dict(pos=A + 4), 4), (dict(B=1 << 20, L=1 << 20), 6),
    (dict(B=0), 0), (dict(L=0), 0), (dict(Hq=0, Hk=0), 0)])
def test_rope_refusals(nat, kw, code):
    assert _rope(nat, **kw) == code


def test_rope_bwd_refusals(nat):
    dm = lambda **kw: nat.RopeDims(1, 4, 2, 1, 64, 64, 0, kw.get("norm", 1), kw.get("dtype", 0), 1e-6)
    s = nat.Strides(512, 256, 64)

    def call(d, g=1, x=0, dw=A, ws=A, nws=1 << 30, dq=A):
        return nat.lib.nats_qk_norm_rope_bwd(d, g, x, A, s, A, s, A, s, A, s, None, None, A, None, 0, 0, dq, s, A, s, dw,
                                             dw, ws, nws, None)

    assert call(dm(), g=7) == 3 and call(dm(), x=-1) == 3
    assert call(dm(dtype=1), g=0, x=1) == 3 and call(dm(dtype=1), g=1, x=0) == 3
    assert call(dm(norm=0)) == 9
    assert call(dm(), dq=None) == 1 and call(dm(), ws=None) == 1
    assert call(dm(), ws=A + 8) == 4
    assert call(dm(), nws=nat.lib.nats_qk_norm_rope_bwd_workspace_size(dm()) - 1) == 5
    bad = nat.RopeDims(1, 4, 2, 1, 65, 64, 0, 1, 0, 1e-6)
    assert nat.lib.nats_qk_norm_rope_bwd_workspace_size(bad) == 0


def _cache(nat, **kw):
    c = dict(k_pages=A, v_pages=A, weight=A, table=A, lens=A + 4, err=A, n_pages=8, page=16, Hk=2, d=64, B=3, max_pages=4,
             dtype=0)
    c.update(kw)
    return nat.PagedCache(*[c[n] for n, _ in nat.PagedCache._fields_])


BAD_CACHE = [(dict(page=24), 2), (dict(page=0), 2), (dict(Hk=0), 2), (dict(B=-1), 2), (dict(n_pages=-1), 2),
             (dict(max_pages=-1), 2), (dict(d=80), 6), (dict(dtype=2), 3), (dict(max_pages=1 << 28), 6),
             (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
             (dict(err=None), 1), (dict(k_pages=A + 8), 4), (dict(lens=A + 2), 4)]


@pytest.mark.parametrize("kw,code", BAD_CACHE)
def test_cache_refusals(nat, kw, code):
    c = _cache(nat, **kw)
    s = nat.Strides(512, 256, 64)
    dm = nat.RopeDims(c.B, 1, 0, c.Hk, c.d, 0, 0, 0, c.dtype, 1e-6)
    # the address of a struct member's NULL is None
    assert nat.lib.nats_paged_decode(c, 4, 0.0, A, 256, 64, A, None, 0, A, 1 << 40, None) == code
    assert nat.lib.nats_paged_append(c, dm, None, None, A, s, A, s, None, None, None, None, None, None, 0, None, None,
                                     None) == code
    assert nat.lib.nats_paged_evict(c, A + 64, 4, 32, 0, 0, A + 128, None, A, 1 << 40, None) == code


def test_decode_refusals(nat):
    c = _cache(nat)

    def call(c=c, Hq=4, scale=0.0, q=A, qb=256, qh=64, out=A, acc=0, ws=A, nws=1 << 40):
        return nat.lib.nats_paged_decode(c, Hq, scale, q, qb, qh, out, None, acc, ws, nws, None)

    assert call(Hq=3) == 2 and call(Hq=-2) == 2
    assert call(scale=-1.0) == 9 and call(scale=float("nan")) == 9
    assert call(q=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
    assert call(c=_cache(nat, weight=None), acc=1) == 1
    assert call(q=A + 8) == 4 and call(qh=65) == 4 and call(qb=4) == 4 and call(out=A + 4) == 4
    need = nat.lib.nats_paged_decode_workspace_size(c, 4, 0)
    assert call(nws=need - 1) == 5
    assert nat.lib.nats_paged_decode_workspace_size(c, 4, 1) >= need + 4 * 3 * 4 * 64
    assert nat.lib.nats_paged_decode_workspace_size(c, 3, 0) == 0
    assert call(Hq=0) == 0 and call(c=_cache(nat, B=0)) == 0


def test_evict_refusals(nat):
    c = _cache(nat)

    def call(c=c, ot=A + 64, pages=4, budget=32, recent=0, sinks=0, lens=A + 128, ws=A, nws=1 << 40):
        return nat.lib.nats_paged_evict(c, ot, pages, budget, recent, sinks, lens, None, ws, nws, None)

    assert call(budget=-1) == 2 and call(budget=65) == 2 and call(pages=-1) == 2
    assert call(recent=-1) == 9 and call(sinks=-1) == 9 and call(recent=30, sinks=3) == 9
    assert call(recent=(1 << 31) - 1, sinks=(1 << 31) - 1) == 9
    assert call(ot=A) == 9 and call(lens=A + 4) == 9
    assert call(ot=None) == 1 and call(lens=None) == 1 and call(ws=None) == 1 and call(c=_cache(nat, weight=None)) == 1
    assert call(ws=A + 8) == 4
    assert call(nws=nat.lib.nats_paged_evict_workspace_size(c, 32) - 1) == 5
    assert call(c=_cache(nat, B=0)) == 0


def test_evict_to_nothing_still_reads_the_weights(nat):
    c = _cache(nat, weight=None)
    assert nat.lib.nats_paged_evict(c, None, 0, 0, 0, 0, A + 128, None, A, 1 << 40, None) == 1


def test_append_refusals(nat):
    c = _cache(nat)
    s = nat.Strides(512, 256, 64)

    def call(c=c, B=3, Hk=2, d=64, dtype=0, Hq=0, rot=0, L=2, q=None, k=A, v=A, f=None, oq=None, start=None):
        dm = nat.RopeDims(B, L, Hq, Hk, d, rot, 0, 0, dtype, 1e-6)
        return nat.lib.nats_paged_append(c, dm, q, s, k, s, v, s, None, None, f, start, None, None, 0, oq, s, None)

    assert call(B=2) == 2 and call(Hk=1) == 2 and call(d=128) == 2 and call(dtype=1) == 3
    assert call(k=None) == 1 and call(v=None) == 1 and call(Hq=2) == 1 and call(rot=64) == 1
    assert call(k=A + 1) == 4 and call(start=A + 1) == 4
    assert call(L=0) == 0


# ------------------------------------------------------------ index models

def _turns_fixed(f):
    """The kernel's integer arithmetic, step by step (csrc/qk_rope.cu turns_fixed)."""
    import struct

    bits = struct.unpack("<Q", struct.pack("<d", f))[0]
    e = (bits >> 52) & 0x7FF
    if e in (0, 0x7FF):
        return 0
    m = (bits & ((1 << 52) - 1)) | (1 << 52)
    prod = m * 2935890503282001226
    lo, hi = prod & ((1 << 64) - 1), prod >> 64
    s = 1075 - e
    if s <= 0:
        r = 0 if -s >= 64 else (lo << -s)
    elif s < 64:
        r = (lo >> s) | (hi << (64 - s))
    else:
        r = 0 if s >= 128 else hi >> (s - 64)
    r &= (1 << 64) - 1
    return (-r) & ((1 << 64) - 1) if bits >> 63 else r


def test_fixed_point_turns():
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    rng = random.Random(1)
    for f in [1.0, 0.5, 10000.0 ** -0.5, 1e-6, 2.5, 1e-20, -0.7] + [10.0 ** rng.uniform(-12, 2) for _ in range(200)]:
        want = Fraction(f) / two_pi * 2 ** 64
        got = _turns_fixed(f)
        diff = (got - want) % 2 ** 64
        diff = min(diff, 2 ** 64 - diff)
        # the constant's rounding (half a unit of its 62 bits) and the shift's truncation
        assert diff <= abs(want) * Fraction(1, 2 ** 61) + 1
    assert _turns_fixed(0.0) == 0 and _turns_fixed(math.inf) == 0 and _turns_fixed(math.nan) == 0


@pytest.mark.parametrize("seed", range(30))
def test_tile_line_is_covered_once_and_joined(seed):
    """The deal of 64-slot tiles to CTAs (csrc/paged_decode.cu): every tile of every unit is taken by one CTA, a unit
    in several runs is found again by the join from the same numbers, and no two partials share a slot."""
    rng = random.Random(seed)
    ctas = rng.choice([1, 7, 152, 456])
    U = rng.choice([1, 3, 8, 16])
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randrange(5000)]) for _ in range(rng.randrange(1, 40))]
    nt = [-(-n // 64) for n in lens]
    pre = [sum(nt[:b]) for b in range(len(nt) + 1)]
    T = pre[-1] * U
    ctas = min(ctas, T, max(32 * U * sum(x > 0 for x in nt), T // 4))  # decode_ctas
    partial, direct = {}, set()
    used = set()
    for c in range(ctas):
        s, e = T * c // ctas, T * (c + 1) // ctas
        cur = s
        b = next((b for b in range(len(nt)) if pre[b] * U <= s < pre[b + 1] * U), 0)
        base = pre[b]
        while cur < e:
            if cur >= (base + nt[b]) * U:
                base += nt[b]
                b += 1
                continue
            u, t0 = divmod(cur - base * U, nt[b])
            t1 = min(nt[b], t0 + e - cur)
            if t0 == 0 and t1 == nt[b]:
                direct.add((b, u))
            else:
                slot = 2 * c + (0 if cur == s else 1)
                assert slot not in used
                used.add(slot)
                partial.setdefault((b, u), []).append((slot, t0, t1))
            cur += t1 - t0
    for b in range(len(nt)):
        for u in range(U):
            if nt[b] == 0:
                continue
            x0 = pre[b] * U + u * nt[b]
            c0, c1 = (((x + 1) * ctas - 1) // T for x in (x0, x0 + nt[b] - 1))
            if c0 == c1:
                assert (b, u) in direct and (b, u) not in partial
                continue
            first = 2 * c0 + (0 if T * c0 // ctas == x0 else 1)
            slots = [first] + [2 * c for c in range(c0 + 1, c1 + 1)]
            got = sorted(partial[(b, u)], key=lambda p: p[1])
            assert [g[0] for g in got] == slots
            assert got[0][1] == 0 and got[-1][2] == nt[b] and all(x[2] == y[1] for x, y in zip(got, got[1:]))


# ------------------------------------------------------------ 64-bit forms

@pytest.mark.parametrize("inter", [False, True])
def test_reference_gradient_against_differences(inter):
    rng = torch.Generator().manual_seed(1)
    x, dy = torch.randn(1, 2, 3, 64, generator=rng).double(), torch.randn(1, 2, 3, 64, generator=rng).double()
    w, pos = 1 + 0.3 * torch.randn(64, generator=rng).double(), torch.tensor([[5, 1000, 31]])
    f = torch.tensor([100.0 ** (-i / 24) for i in range(24)], dtype=torch.float64)
    dx, dw, _ = ref.norm_rotate_bwd(dy, x, w, pos, f, inter, True, 1e-6)
    fwd = lambda a, b: (dy * ref.norm_rotate(a, b, pos, f, inter, True, 1e-6)).sum()
    for _ in range(5):
        v, vw = torch.randn(x.shape, generator=rng).double(), torch.randn(64, generator=rng).double()
        h = 1e-5
        assert abs((fwd(x + h * v, w) - fwd(x - h * v, w)) / (2 * h) - (dx * v).sum()) < 1e-7
        assert abs((fwd(x, w + h * vw) - fwd(x, w - h * vw)) / (2 * h) - (dw * vw).sum()) < 1e-7


def test_reference_decode_is_a_softmax_over_the_used_slots():
    rng = torch.Generator().manual_seed(2)
    table = torch.tensor([[2, 0], [1, -1]], dtype=torch.int32)
    k, v = torch.randn(3, 2, 16, 64, generator=rng).double(), torch.randn(3, 2, 16, 64, generator=rng).double()
    q = torch.randn(2, 4, 64, generator=rng).double()
    ref.HALF.setdefault(torch.float64, 0.0)
    out, lse, ps, _, _ = ref.decode(q, k, v, table, [20, 3])
    rows = torch.cat([k[2, 1], k[0, 1, :4]]), torch.cat([v[2, 1], v[0, 1, :4]])
    p = torch.softmax(rows[0] @ q[0, 3] / 8, 0)
    assert torch.allclose(out[0, 3], p @ rows[1], rtol=0, atol=1e-12) and torch.allclose(ps[0][1, 1], p)
    assert abs(float(lse[0, 3]) - float(torch.logsumexp(rows[0] @ q[0, 3] / 8, 0)) / math.log(2)) < 1e-12
