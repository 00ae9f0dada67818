"""The paged decode's arithmetic where an ordinary error bound would hide a loss:
scores that the products form exactly, so that what is left are the softmax's
own roundings, against 64 bits."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def nats():
    from linear_attention_nats_gb300 import build

    build.build()
    import linear_attention_nats_gb300 as n

    return n


def _shared(nats, k, v, B, n, page, weight=None):
    """B sequences over the same pages, which hold k, v [Hk, n, d] in order."""
    pages = lambda x: x.unflatten(1, (-1, page)).transpose(0, 1).contiguous()
    table = torch.arange(k.shape[1] // page, dtype=torch.int32).repeat(B, 1)
    return nats.PagedCache(pages(k).cuda(), pages(v).cuda(), table.cuda(),
                           torch.full((B,), n, dtype=torch.int32).cuda(), weight=weight)


def _settled(x, e):
    """Entries whose rounding to bf16 an error of e cannot change: those further than e from a border between two."""
    lo, hi = (x - e).to(F32).to(BF), (x + e).to(F32).to(BF)
    return lo == hi


# A weight 2^x, x = scale log2 e s - maximum with |x| <= 6: log2 e as fp32 (U of x), the sum's rounding (U of x) and the
# exponential's 2^-22: (12 ln 2 + 4) U < 13 U.  What the sums of weights and values add is stated where it is used.
WEIGHT = 13 * U


@pytest.mark.parametrize("d", [64, 128])
def test_bf16_output_of_two_slots_is_the_rounded_value(nats, d):
    """Two slots with weights 1 and p: out = (v1 + p v2) / (1 + p) with p to nearly all of its fp32, v2 through every
    significand.  Above the weights' own error: the products and sums of a step (6 steps cut off at 2^-23, of the
    weighted magnitudes), the sum's three additions, the quotient and the product: 18 U."""
    B = 1500
    rng = torch.Generator().manual_seed(1)
    q = torch.zeros(B, 1, d)
    q[:, 0, 0] = (torch.rand(B, generator=rng) + 0.5).to(BF).float()
    k = torch.zeros(1, 16 * B, d)
    k[0, 1::16, 0] = -4 * torch.rand(B, generator=rng).to(BF).float()
    v = torch.zeros(1, 16 * B, d)
    v[0, 1::16] = (1 + torch.randint(0, 128, (B, d), generator=rng) / 128.0)
    pages = lambda x: x.unflatten(1, (-1, 16)).transpose(0, 1).contiguous().to(BF).cuda()
    c = nats.PagedCache(pages(k), pages(v), torch.arange(B, dtype=torch.int32)[:, None].cuda(),
                        torch.full((B,), 2, dtype=torch.int32).cuda())
    out = nats.paged_decode(c, q.to(BF).cuda(), scale=1.0).cpu()[:, 0]
    p = torch.exp(q[:, 0, 0].double() * k[0, 1::16, 0].to(BF).double())[:, None]
    v2 = v[0, 1::16].double()
    e = p * v2 / (1 + p)
    bound = WEIGHT * p * (v2 - e) / (1 + p) + 18 * U * e
    sure = _settled(e, bound)
    assert sure.double().mean() > 0.99
    assert torch.equal(out[sure], e.to(BF)[sure])


@pytest.mark.parametrize("d", [64, 128])
def test_bf16_output_of_many_steps_of_one_cta_is_the_rounded_value(nats, d):
    """A unit that one CTA takes from end to end, 65,536 slots, with weights and values of one sign, so that errors that
    lean one way would add up.  A lane's sum takes 1024 rounded additions and the values' 64 between their runs of 16
    steps: errors of either sign, taken as independent (Higham and Mary, 2019: lambda sqrt(n) U, lambda = 6), 6 (32 + 8)
    U.  Within a run three products a step are cut off at 2^-23 of a sum that grows to the run's own: 48 x 2^-23 at
    most.  Joins, quotient and product: 20 U."""
    n, page, B = 65536, 64, 152 * (4 if d == 64 else 3)
    rng = torch.Generator().manual_seed(2)
    k = torch.zeros(1, n, d)
    k[0, :, 0] = -torch.rand(n, generator=rng)
    share = torch.linspace(0.02, 0.98, d)
    v = torch.where(torch.rand(n, d, generator=rng) < share, 1.0, 2 - 2.0 ** -7)[None]
    q = torch.zeros(B, 1, d)
    q[:, 0, 0] = 0.5 + torch.rand(B, generator=rng)
    k, v, q = k.to(BF), v.to(BF), q.to(BF)
    out = nats.paged_decode(_shared(nats, k, v, B, n, page), q.cuda(), scale=1.0).cpu()[:, 0]
    p = torch.softmax((q[:, 0, :1].double().cuda() @ k[0, :, :1].double().cuda().T), -1)
    e = (p @ v[0].double().cuda()).cpu()
    bound = (WEIGHT * 0.5 + (6 * 40 + 48 * 2 + 20) * U) * e  # (values within half of e of it)
    sure = _settled(e, bound)
    assert sure.double().mean() > 0.95
    assert torch.equal(out[sure], e.to(BF)[sure])


@pytest.mark.parametrize("G,d", [(1, 64), (1, 128), (12, 64), (12, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_maximum_that_rises_through_a_long_run(nats, G, d, dtype):
    """Scores that rise by some 90 powers of two over a CTA's run, now slowly, now in jumps, so that the sums of all
    earlier steps are rescaled again and again; heads of one group rise at different places."""
    n, page, B = 8192, 64, 640
    rng = torch.Generator().manual_seed(3)
    k = torch.zeros(1, n, d)
    k[0, :, 0] = torch.linspace(-60, 0, n)
    k[0, :, 1] = torch.where(torch.arange(n) < 5000, -40.0, 0.0)
    k[0, :, 2] = -50.0 * torch.rand(n, generator=rng) * (torch.arange(n) % 700 != 1)
    v = torch.randn(1, n, d, generator=rng)
    q = torch.zeros(B, G, d)
    for h in range(G):
        q[:, h, h % 3] = 1.0
    q[:, :, 3] = torch.randn(B, 1, generator=rng)
    k[0, :, 3] = torch.randn(n, generator=rng)
    k, v, q = k.to(dtype), v.to(dtype), q.to(dtype)
    out = nats.paged_decode(_shared(nats, k, v, B, n, page), q.cuda(), scale=1.0).cpu().double()
    qd, kd, vd = q.double().cuda(), k[0].double().cuda(), v[0].double().cuda()
    s = qd @ kd.T
    p = torch.softmax(s, -1)
    e, mag = (p @ vd).cpu(), (p @ vd.abs()).cpu()
    # a score: four products and their sum, each off by 2^-23 of |q| |k| <= 70, and its scaling: 8 x 2^-23 x 70; the
    # weights that count lie within 20 of the maximum; sums as above, all steps' signs alike: (4 x 128 / 4 + 64) 2^-23
    rel = 2 * (8 * 70 * 2.0 ** -23 + 20 * 2 * U + 4 * U) + (128 + 64) * 2.0 ** -23
    half = 2.0 ** -8 if dtype == BF else U
    assert ((out - e).abs() <= half * (e.abs() + rel * mag) + rel * mag).all()


@pytest.mark.parametrize("n,w0", [(64, 2.0 ** 20), (4096, 2.0 ** 14), (50, 3e5), (4000, 1000.0)])
@pytest.mark.parametrize("G,dtype", [(8, BF), (8, F32), (24, BF)])
def test_weights_of_heavy_slots_grow_by_the_groups_sum(nats, n, w0, G, dtype):
    """Equal scores: each head gives every slot 1 / n, which of a heavy slot's weight is less than half a step, the
    group's G / n is not.  One rounding a call (U of the weight), and the group's own sum: G + 8 roundings."""
    calls, page, d = 64, 16, 64
    N = -(-n // page) * page
    weight = torch.full((N // page, 1, page), w0, device="cuda")
    c = _shared(nats, torch.zeros(1, N, d, dtype=dtype), torch.ones(1, N, d, dtype=dtype), 1, n, page, weight)
    q = torch.zeros(1, G, d, dtype=dtype, device="cuda")
    for _ in range(calls):
        nats.paged_decode(c, q, accumulate=True)
    got = c.weight.cpu().double().reshape(-1)
    want = w0 + calls * G / n
    assert ((got[:n] - want).abs() <= calls * (U * want * (1 + U) + (G + 8) * U * G / n)).all()
    assert (got[n:] == w0).all()


@pytest.mark.parametrize("n", [50, 1000, 9000])
@pytest.mark.parametrize("G,dtype", [(1, BF), (4, F32), (9, BF), (9, F32)])
def test_weights_of_large_scores(nats, n, G, dtype):
    """Scores of about 4096 (5909 in powers of two, where fp32 has steps of 2^-11) that lie close together and that the
    products form exactly: the weights go by their distances.  A weight is off by WEIGHT where its distance counts
    (|x| <= 12 doubles it), its sum by 64 + n / 4 roundings of positive numbers, its quotient by 2 U, the group's sum by
    G U, and the stored one by its own rounding."""
    page, d = 16, 64
    N = -(-n // page) * page
    rng = torch.Generator().manual_seed(5)
    k = torch.zeros(1, N, d)
    k[0, :, 0] = 4096
    k[0, :, 1] = -torch.randint(0, 65, (N,), generator=rng) / 8.0
    q = torch.zeros(1, G, d)
    q[:, :, :2] = 1
    c = _shared(nats, k.to(dtype), torch.randn(1, N, d, generator=rng).to(dtype), 1, n, page,
                torch.zeros(N // page, 1, page, device="cuda"))
    nats.paged_decode(c, q.to(dtype).cuda(), scale=1.0, accumulate=True)
    want = G * torch.softmax((k[0, :n, 0] + k[0, :n, 1]).double(), -1)
    got = c.weight.cpu().double().reshape(-1)[:n]
    assert ((got - want).abs() <= (4 * WEIGHT + (64 + n / 4 + 2 + G + 1) * U) * want).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_sequence_inside_wider_rows(nats, dtype):
    """One sequence whose rows lie in a matrix of an odd width: the stride between sequences says nothing."""
    rng = torch.Generator().manual_seed(6)
    Hq, Hk, d, n = 4, 2, 64, 40
    rows = torch.randn(3, (Hq + 2 * Hk) * d + 3, generator=rng).to(dtype).cuda()
    q, k, v = (rows.as_strided((1, b - a, d), (rows.stride(0), d, 1), a * d) for a, b in ((0, 4), (4, 6), (6, 8)))
    assert q.is_contiguous() and q.stride(0) % 2 == 1
    f = nats.rope_inv_freq(d)
    got = []
    for copy in (lambda t: t, lambda t: torch.empty(t.shape, dtype=dtype, device="cuda").copy_(t)):
        c = nats.PagedCache.empty(4, 16, Hk, d, 1, 4, dtype=dtype)
        c.table.copy_(torch.arange(4, dtype=torch.int32)[None])
        x = [copy(t)[:, :, None] for t in (q, k, v)]
        for _ in range(n):
            oq = nats.paged_append(c, x[1], x[2], q=x[0], norm=True, inv_freq=f)
            c.lens.add_(1)
        r = nats.qk_norm_rope(x[0], x[1], None, None, f, pos0=n - 1)
        g = nats.qk_norm_rope_bwd(*r, x[0], x[1], None, None, f, pos0=n - 1)
        got.append([nats.paged_decode(c, copy(q)), oq, c.k_pages, c.v_pages, *r, *g.values()])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("Hk,G,d,dtype", [(2, 4, 128, BF), (1, 9, 64, BF), (3, 1, 64, F32), (2, 12, 128, F32), (1, 40, 64, BF)])
def test_weights_under_tables_longer_than_the_pool(nats, Hk, G, d, dtype):
    """Tables for contexts far longer than the pool: what a call gives is what it gives with tables that just fit, bad
    entries and the pool's last page among them."""
    rng = torch.Generator().manual_seed(7 + G)
    page, lens = 16, [700, 33, 0, 1, 64, 200]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need)
    shape = (n_pages, Hk, page, d)
    k, v, w0 = torch.randn(shape, generator=rng), torch.randn(shape, generator=rng), torch.rand(shape[:3], generator=rng)
    q = torch.randn(len(lens), Hk * G, d, generator=rng).to(dtype).cuda()
    order, at, rows = torch.randperm(n_pages, generator=rng).int(), 0, []
    for m in need:
        rows.append(order[at:at + m].tolist())
        at += m
    rows[0][5], rows[1][1], rows[5][0] = -1, n_pages, -5
    got = []
    for width in (max(need), 40 * n_pages):
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        for b, r in enumerate(rows):
            table[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
        c = nats.PagedCache(k.to(dtype).cuda(), v.to(dtype).cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            weight=w0.cuda())
        ws = torch.full((nats.paged_workspace_size(c, Hq=Hk * G, accumulate=True),), 255, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            out, lse = nats.paged_decode(c, q, accumulate=True, return_lse=True, workspace=ws)
        got.append((out, lse, c.weight))
        with pytest.raises(nats.NatsError):
            c.check()
    tight, wide = got
    if dtype == F32 and G > 8:
        # the wide table's units are of sixteen heads: other sums, the same values.  A score of either is off by (d + 8)
        # 2^-23 of scale |q| |k|, a factor by twice that (its maximum too), outputs and weights by twice a factor's
        score = (d + 8) * 2.0 ** -23 * d ** -0.5 * float(q.norm(dim=-1).max()) * float(k.norm(dim=-1).max())
        tol = 2 * 4 * score * max(1.0, float(v.abs().max()))
        for a, b in zip(tight, wide):
            fin = torch.isfinite(a)
            assert torch.equal(fin, torch.isfinite(b)) and ((a - b)[fin].abs() <= tol * (1 + a[fin].abs())).all()
    else:
        assert all(torch.equal(a, b) for a, b in zip(tight, wide))
    # every sequence's weights sum to its query heads (the slots of bad entries have none)
    per = sum(Hk * G for n in lens if n)
    assert abs(float(wide[2].double().sum() - w0.double().sum()) - 2 * per) < 1e-3 * per


def test_scale_too_small_for_its_type_is_refused(nats):
    """It would be taken as 0, which asks for 1 / sqrt(d)."""
    c = nats.PagedCache.empty(2, 16, 1, 64, 1, 2)
    q = torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    for scale in (1e-60, -1e-60):
        with pytest.raises(ValueError):
            nats.paged_decode(c, q, scale=scale)
    nats.paged_decode(c, q, scale=1e-40)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_reach_no_further_than_a_nan(nats, dtype):
    """An infinite value reaches its entry of its group's rows, an infinite key its group's rows and weights; all else
    keeps its bits."""
    rng = torch.Generator().manual_seed(8)
    n, Hk, G, d, page = 300, 2, 3, 64, 16
    pages = -(-n // page)
    k, v = (torch.randn(pages, Hk, page, d, generator=rng).to(dtype) for _ in range(2))
    q = torch.randn(1, Hk * G, d, generator=rng).to(dtype).cuda()

    def run(k, v):
        c = nats.PagedCache(k.cuda(), v.cuda(), torch.arange(pages, dtype=torch.int32)[None].cuda(),
                            torch.tensor([n], dtype=torch.int32).cuda(), weight=torch.ones(pages, Hk, page, device="cuda"))
        return nats.paged_decode(c, q, accumulate=True).cpu(), c.weight.cpu()

    out, w = run(k, v)
    for x in (math.inf, -math.inf):
        bad = v.clone()
        bad[3, 0, 5, 7] = x
        o, u = run(k, bad)
        assert not torch.isfinite(o[0, :G, 7]).any() and torch.equal(u, w)
        o[0, :G, 7] = out[0, :G, 7]
        assert torch.equal(o, out)
        bad = k.clone()
        bad[3, 1, 5, 7] = x
        o, u = run(bad, v)
        assert torch.equal(o[0, :G], out[0, :G]) and torch.equal(u[:, 0], w[:, 0])


@pytest.mark.parametrize("n", [60, 3000])
@pytest.mark.parametrize("G,dtype", [(2, BF), (2, F32), (12, BF), (12, F32)])
def test_scores_up_to_the_stated_size(nats, n, G, dtype):
    """Scores near 2^27 (2^27.5 in powers of two: steps of 16) that the products form exactly and that rise slot by slot:
    outputs and weights go by their distances, multiples of 8.  Bounds as above, a weight's for its own distance x: (2 |x|
    ln 2 + 4) U, and 2^-126 where fp32's exponential ends; the outputs of n / 16 steps: (n / 4 + 64) 2^-23 of the weighted
    magnitudes, what is more than 12 away counting for nothing."""
    page, d = 16, 64
    N = -(-n // page) * page
    rng = torch.Generator().manual_seed(9)
    k = torch.zeros(1, N, d)
    k[0, :, 0] = 2.0 ** 27
    k[0, :n, 1] = -8.0 * torch.randint(0, 32, (n,), generator=rng).sort(descending=True).values
    q = torch.zeros(1, G, d)
    q[:, :, :2] = 1
    v = torch.randn(1, N, d, generator=rng).to(dtype)
    c = _shared(nats, k.to(dtype), v, 1, n, page, torch.zeros(N // page, 1, page, device="cuda"))
    out, lse = nats.paged_decode(c, q.to(dtype).cuda(), scale=1.0, accumulate=True, return_lse=True)
    p = torch.softmax((k[0, :n, 0].double() + k[0, :n, 1].double()), -1)
    got = c.weight.cpu().double().reshape(-1)[:n]
    x = (k[0, :n, 1].double().max() - k[0, :n, 1].double()) * math.log2(math.e)
    rel = (2 * x * math.log(2) + 4) * U + 2 * WEIGHT + (64 + n / 4 + 2 + G + 1) * U
    assert ((got - G * p).abs() <= rel * G * p + G * 2.0 ** -126).all()
    e, mag = p @ v[0, :n].double(), p @ v[0, :n].double().abs()
    rel = 8 * WEIGHT + (n / 4 + 64) * 2.0 ** -23
    half = 2.0 ** -8 if dtype == BF else U
    assert ((out.cpu().double()[0] - e).abs() <= half * (e.abs() + rel * mag) + rel * mag).all()
    assert ((lse.cpu().double() - 2.0 ** 27 * math.log2(math.e)).abs() <= 16).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_most_heads_a_group(nats, dtype):
    """4096 query heads on one key head, with weights: sums and factors of a whole group in shared memory."""
    import serving_ref as ref

    rng = torch.Generator().manual_seed(10)
    lens, page, d, G = [200, 10, 0], 16, 64, 4096
    table, _, n_pages = ref.assign(lens, page, rng)
    k, v = (torch.randn(n_pages, 1, page, d, generator=rng).to(dtype) for _ in range(2))
    q = torch.randn(len(lens), G, d, generator=rng).to(dtype)
    c = nats.PagedCache(k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                        weight=torch.zeros(n_pages, 1, page, device="cuda"))
    out = nats.paged_decode(c, q.cuda(), accumulate=True)
    e, _, ps, err, perr = ref.decode(q, k, v, table, lens)
    assert ((out.cpu().double() - e).abs() <= ref.HALF[dtype] * (e.abs() + err) + err).all()
    got = c.weight.cpu().double()
    for b, n in enumerate(lens):
        w, want = ref.slots(got, table, b, n, page)[0], ps[b].sum(1)[0]
        assert ((w - want).abs() <= perr[b].sum(1)[0] + (G + 1) * U * want).all()
