"""The paged key / value cache - append, attention of one new token, eviction
- against plain 64-bit forms."""

import math

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


def _pool(rng, n_pages, Hk, page, d, dtype, garbage=True):
    """Pages whose unused rows hold NaN and infinities (the caller fills the used ones)."""
    k = torch.full((n_pages, Hk, page, d), math.nan if garbage else 0.0).to(dtype)
    v = torch.full((n_pages, Hk, page, d), math.inf if garbage else 0.0).to(dtype)
    return k, v


def _filled(rng, lens, page, Hk, d, dtype, extra=0):
    table, spare, n_pages = ref.assign(lens, page, rng, extra)
    k, v = _pool(rng, n_pages, Hk, page, d, dtype)
    for b, n in enumerate(lens):
        j = torch.arange(int(n))
        at = table[b].long()[j // page]
        k[at, :, j % page] = torch.randn(int(n), Hk, d, generator=rng).to(dtype)
        v[at, :, j % page] = torch.randn(int(n), Hk, d, generator=rng).to(dtype)
    return table, spare, k, v


def _cache(nats, table, lens, k, v, weight=None):
    return nats.PagedCache(k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                           weight=None if weight is None else weight.cuda())


# ------------------------------------------------------------------ decode

DECODE = [
    # lens, Hk, G, d, page, dtype
    ([1], 1, 1, 64, 16, BF),
    ([0], 2, 3, 128, 16, F32),
    ([517], 16, 1, 128, 64, BF),
    ([64, 63, 65, 0, 1], 2, 4, 128, 64, BF),
    ([100, 0, 257, 16, 15, 17], 3, 2, 64, 48, F32),
    ([300, 7], 1, 5, 128, 32, BF),
    ([129, 2048], 2, 8, 64, 128, BF),
    ([700, 31, 0, 0, 400], 2, 12, 128, 16, BF),
    ([333, 95], 1, 16, 128, 64, BF),
    ([210], 1, 24, 64, 16, F32),
    ([9000, 3], 2, 3, 128, 16, F32),
    ([20000], 1, 7, 128, 64, BF),
    ([130, 50, 0, 1000], 1, 40, 64, 16, BF),
    ([257, 64], 2, 20, 128, 32, F32),
    ([5000, 300], 1, 32, 128, 64, BF),
    ([3] * 150 + [200] + [0] * 40, 1, 2, 64, 16, BF),
]


@pytest.mark.parametrize("lens,Hk,G,d,page,dtype", DECODE)
@pytest.mark.parametrize("accumulate", [False, True])
def test_decode(nats, lens, Hk, G, d, page, dtype, accumulate):
    rng = torch.Generator().manual_seed(len(lens) * 100 + G)
    table, _, k, v = _filled(rng, lens, page, Hk, d, dtype)
    B, Hq = len(lens), Hk * G
    q = (2 * torch.randn(B, Hq, d, generator=rng)).to(dtype)
    w0 = torch.rand(k.shape[:3], generator=rng)
    c = _cache(nats, table, lens, k, v, w0 if accumulate else None)
    out, lse = nats.paged_decode(c, q.cuda(), accumulate=accumulate, return_lse=True)
    e, elog, ps, err, perr = ref.decode(q, k, v, table, lens)
    diff = (out.cpu().double() - e).abs()
    assert (diff <= ref.HALF[dtype] * (e.abs() + err) + err).all()
    empty = torch.isinf(elog)
    assert torch.equal(torch.isinf(lse.cpu()), empty) and (lse.cpu()[empty] < 0).all()
    # log2 of a sum of factors each off by the p's own relative bound, then rounded
    fin = ~empty
    assert ((lse.cpu().double() - elog)[fin].abs() <= 2.0 ** -22 * elog[fin].abs() + (d + 8) * 2.0 ** -20 + 1e-5).all()
    c.check()
    if accumulate:
        want, tol = w0.double(), torch.zeros(w0.shape, dtype=torch.float64)
        for b, n in enumerate(lens):
            j = torch.arange(n)
            at = table[b].long()[j // page]
            want[at, :, j % page] += ps[b].sum(1).T
            tol[at, :, j % page] += perr[b].sum(1).T
        got = c.weight.cpu().double()
        assert ((got - want).abs() <= tol + ref.U * (want.abs() * 2 + G)).all()
        assert torch.equal(got[tol == 0], want[tol == 0])


# groups of more than eight fp32 heads in tables of many tiles: units of sixteen
@pytest.mark.parametrize("Hk,G,d", [(2, 12, 64), (2, 12, 128), (1, 16, 128), (1, 35, 64), (3, 9, 128)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_decode_wide_groups_of_many_sequences(nats, Hk, G, d, accumulate):
    lens = [1024, 0, 1000, 64, 65, 1] + [(7 * i) % 200 for i in range(94)]
    test_decode(nats, lens, Hk, G, d, 64, F32, accumulate)


def test_decode_strided_query_scale_and_out(nats):
    rng = torch.Generator().manual_seed(1)
    lens = [70, 5, 130]
    table, _, k, v = _filled(rng, lens, 16, 2, 64, BF)
    wide = torch.randn(3, 6, 3, 64, generator=rng).to(BF).cuda()
    q = wide[:, :, 1]
    c = _cache(nats, table, lens, k, v)
    out = torch.full((3, 6, 64), 5.0, dtype=BF, device="cuda")
    assert nats.paged_decode(c, q, scale=0.05, out=out) is out
    e, _, _, err, _ = ref.decode(q.cpu(), k, v, table, lens, scale=0.05)
    assert ((out.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()


def test_decode_repeats_bit_for_bit_and_shares_pages(nats):
    """Two sequences over the same pages get the same bits, whatever their place in the line of tiles."""
    rng = torch.Generator().manual_seed(2)
    table, _, k, v = _filled(rng, [1000], 64, 2, 128, BF)
    q = torch.randn(1, 8, 128, generator=rng).to(BF)
    c = _cache(nats, table.repeat(2, 1), [1000, 1000], k, v)
    a = nats.paged_decode(c, q.repeat(2, 1, 1).cuda())
    b = nats.paged_decode(c, q.repeat(2, 1, 1).cuda())
    assert torch.equal(a, b)
    e, _, _, err, _ = ref.decode(q, k, v, table, [1000])
    assert ((a.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_leaves_out_bad_pages_and_reports_them(nats, dtype):
    rng = torch.Generator().manual_seed(3)
    lens, page = [100, 80], 16
    table, _, k, v = _filled(rng, lens, page, 2, 64, dtype)
    bad = table.clone()
    bad[0, 2], bad[1, 0] = k.shape[0], -7  # slots 32..47 of sequence 0, 0..15 of sequence 1
    skip = [(0, j) for j in range(32, 48)] + [(1, j) for j in range(16)]
    w0 = torch.rand(k.shape[:3], generator=rng)
    c = _cache(nats, bad, lens, k, v, w0)
    q = torch.randn(2, 8, 64, generator=rng).to(dtype)
    out = nats.paged_decode(c, q.cuda(), accumulate=True)
    e, _, _, err, _ = ref.decode(q, k, v, table, lens, skip=skip)
    assert ((out.cpu().double() - e).abs() <= ref.HALF[dtype] * (e.abs() + err) + err).all()
    with pytest.raises(nats.NatsError):
        c.check()
    skipped = torch.stack([table[0, 2], table[1, 0]]).long()
    assert torch.equal(c.weight.cpu()[skipped], w0[skipped])


@pytest.mark.parametrize("lens,Hk,G,dtype", [([40, 60, 10, 64, 64], 2, 4, BF), ([40, 60, 10, 64, 64], 1, 12, BF),
                                             ([50], 1, 3, F32), ([33, 48, 64, 17, 130, 20], 2, 12, F32)])
def test_decode_weights_of_single_tiles_with_bad_pages(nats, lens, Hk, G, dtype):
    """Sequences of one tile, alone or in a row: the weights of the slots that count, twice over, and no others'."""
    rng = torch.Generator().manual_seed(18 + G)
    page, d = 16, 64
    table, _, k, v = _filled(rng, lens, page, Hk, d, dtype)
    bad = table.clone()
    bad[0, 1] = -1  # slots 16..31 of sequence 0
    skip = [(0, j) for j in range(16, 32)]
    w0 = torch.rand(k.shape[:3], generator=rng)
    c = _cache(nats, bad, lens, k, v, w0)
    q = torch.randn(len(lens), Hk * G, d, generator=rng).to(dtype)
    for _ in range(2):
        out = nats.paged_decode(c, q.cuda(), accumulate=True)
    e, _, ps, err, perr = ref.decode(q, k, v, table, lens, skip=skip)
    assert ((out.cpu().double() - e).abs() <= ref.HALF[dtype] * (e.abs() + err) + err).all()
    want, tol = w0.double(), torch.zeros(w0.shape, dtype=torch.float64)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        at = table[b].long()[j // page]
        want[at, :, j % page] += 2 * ps[b].sum(1).T
        tol[at, :, j % page] += 2 * perr[b].sum(1).T
    got = c.weight.cpu().double()
    # two rounds of G additions to a sum of at most 1 + 2 G
    assert ((got - want).abs() <= tol + 2 * ref.U * (want.abs() * 2 + 2 * G)).all()
    assert torch.equal(c.weight.cpu()[table[0, 1].long()], w0[table[0, 1].long()])


def test_decode_lengths_out_of_range(nats):
    rng = torch.Generator().manual_seed(4)
    table, _, k, v = _filled(rng, [64, 64], 16, 1, 64, BF)
    q = torch.randn(2, 4, 64, generator=rng).to(BF)
    c = _cache(nats, table, [1000, -3], k, v)  # taken as 64 and 0
    out = nats.paged_decode(c, q.cuda())
    e, _, _, err, _ = ref.decode(q, k, v, table, [64, 0])
    assert ((out.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()
    with pytest.raises(nats.NatsError):
        c.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_values_that_are_not_finite(nats, dtype):
    """Such values in slots behind a sequence do not matter (every other test has them there); a NaN in a used slot of
    one key head reaches that head's queries alone: of a value, its entry; of a key, all."""
    rng = torch.Generator().manual_seed(5)
    q = torch.randn(1, 4, 64, generator=rng).to(dtype).cuda()
    for bits in (math.nan, -math.nan):
        table, _, k, v = _filled(rng, [50], 16, 2, 64, dtype)
        v[table[0, 1].long(), 0, 3, 7] = bits
        bad = torch.isnan(nats.paged_decode(_cache(nats, table, [50], k, v), q).cpu())
        assert bad[0, :2, 7].all() and bad.sum() == 2
        table, _, k, v = _filled(rng, [50], 16, 2, 64, dtype)
        k[table[0, 2].long(), 1, 5, 11] = bits
        bad = torch.isnan(nats.paged_decode(_cache(nats, table, [50], k, v), q).cpu())
        assert bad[0, 2:].all() and not bad[0, :2].any()


def test_decode_peaked_scores(nats):
    """One slot that takes nearly everything, and scores far below it."""
    rng = torch.Generator().manual_seed(6)
    for dtype in (BF, F32):
        table, _, k, v = _filled(rng, [400], 16, 1, 128, dtype)
        q = torch.randn(1, 4, 128, generator=rng).to(dtype)
        k[table[0, 11].long(), 0, 5] = 20 * q[0, 0]
        c = _cache(nats, table, [400], k, v)
        out = nats.paged_decode(c, q.cuda())
        e, _, _, err, _ = ref.decode(q, k, v, table, [400])
        assert ((out.cpu().double() - e).abs() <= ref.HALF[dtype] * (e.abs() + err) + err).all()


def test_decode_beyond_32_bit_offsets(nats):
    """A pool of more than 2^31 entries: its last pages hold the sequence."""
    Hk, page, d = 8, 128, 128
    n_pages = (1 << 31) // (Hk * page * d) + 40
    rng = torch.Generator().manual_seed(7)
    k = torch.empty((n_pages, Hk, page, d), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    w = torch.empty((n_pages, Hk, page), device="cuda")
    table = torch.arange(n_pages - 1, n_pages - 25, -1, dtype=torch.int32)[None]
    lens = [24 * page - 5]
    kk, vv = torch.randn(24, Hk, page, d, generator=rng).to(BF), torch.randn(24, Hk, page, d, generator=rng).to(BF)
    k[-24:], v[-24:], w[-24:] = kk.cuda(), vv.cuda(), 0
    c = nats.PagedCache(k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), weight=w)
    q = torch.randn(1, 16, d, generator=rng).to(BF)
    out = nats.paged_decode(c, q.cuda(), accumulate=True)
    small = (table - (n_pages - 24)).int()
    e, _, ps, err, perr = ref.decode(q, kk, vv, small, lens)
    assert ((out.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()
    assert abs(float(w[-24:].double().sum()) - 16) < 1e-3
    # a token appended there
    x = torch.randn(1, Hk, 3, d, generator=rng).to(BF).cuda()
    nats.paged_append(c, x, 2 * x, start=torch.tensor([100], dtype=torch.int32).cuda())
    assert torch.equal(k[-1, :, 100:103], x[0]) and torch.equal(v[-1, :, 100:103], 2 * x[0])
    kk[-1, :, 100:103], vv[-1, :, 100:103] = x[0].cpu(), 2 * x[0].cpu()
    assert (w[-1, :, 100:103] == 0).all()
    # eviction within it: from the last pages to the ones before them
    outt = torch.arange(n_pages - 40, n_pages - 32, dtype=torch.int32)[None].cuda()
    keep, n = nats.paged_evict(c, outt, 8 * page, recent=17, sinks=4, return_keep=True)
    want = ref.evict(w[-24:].cpu(), small, lens, page, 8 * page, 17, 4)
    assert torch.equal(keep.cpu(), want)
    i = torch.arange(8 * page)
    for h in range(Hk):
        src = want[0, h].long()
        assert torch.equal(k[n_pages - 40:n_pages - 32, h].reshape(-1, d).cpu(), kk[small[0].long()[src // page], h, src % page])
        assert torch.equal(v[n_pages - 40:n_pages - 32, h].reshape(-1, d).cpu(), vv[small[0].long()[src // page], h, src % page])


def test_decode_on_another_stream_and_captured(nats):
    rng = torch.Generator().manual_seed(8)
    lens = [300, 40, 0, 1000]
    table, _, k, v = _filled(rng, lens, 16, 2, 64, BF)
    c = _cache(nats, table, lens, k, v, torch.zeros(k.shape[:3]))
    q = torch.randn(4, 6, 64, generator=rng).to(BF).cuda()
    want = nats.paged_decode(c, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nats.paged_decode(c, q, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = nats.paged_decode(c, q, accumulate=True)
    q.copy_(torch.randn(4, 6, 64, generator=rng).to(BF))
    c.lens.copy_(torch.tensor([17, 640, 3, 900], dtype=torch.int32).clamp(max=c.max_pages * 16))
    lens2 = [17, 40, 0, 900]  # pages only hold these; the rest of the table is -1
    c.lens.copy_(torch.tensor(lens2, dtype=torch.int32))
    c.weight.zero_()
    g.replay()
    e, _, _, err, _ = ref.decode(q.cpu(), k, v, table, lens2)
    assert ((out.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()
    assert torch.equal(out, nats.paged_decode(c, q))
    # every sequence's weights sum to its query heads
    assert abs(float(c.weight.double().sum()) - 3 * 6) < 1e-4


def test_decode_calls_in_a_row_share_a_workspace(nats):
    """Calls behind one another on one stream, with one workspace and lengths that change between them, each give
    what they give alone; so do two calls at once on two streams with a workspace each."""
    rng = torch.Generator().manual_seed(13)
    table, _, k, v = _filled(rng, [1500, 700, 900, 64], 16, 2, 128, BF)
    c = _cache(nats, table, [1500, 700, 900, 64], k, v, torch.zeros(k.shape[:3]))
    all_lens = [[1500, 700, 900, 64], [3, 0, 900, 1], [0, 0, 0, 0], [1499, 1, 17, 33], [64, 640, 128, 64]]
    lens = [torch.tensor(x, dtype=torch.int32).cuda() for x in all_lens]
    qs = [torch.randn(4, 10, 128, generator=rng).to(BF).cuda() for _ in lens]
    alone = []
    for q, n in zip(qs, lens):
        c.lens.copy_(n)
        alone.append(nats.paged_decode(c, q))
        torch.cuda.synchronize()
    ws = torch.empty(nats.paged_workspace_size(c, Hq=10, accumulate=True), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(40):
        c.lens.copy_(lens[i % 5])
        got.append(nats.paged_decode(c, qs[i % 5], workspace=ws, accumulate=i % 2 == 1))
    assert all(torch.equal(x, alone[i % 5]) for i, x in enumerate(got))
    weights = sum(10 * sum(n > 0 for n in all_lens[i % 5]) for i in range(1, 40, 2))
    assert abs(float(c.weight.double().sum()) - weights) < 1e-3
    c.lens.copy_(lens[0])
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    both = [nats.paged_decode(c, qs[0], stream=s[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, alone[0]) for x in both)


def test_outputs_of_another_stream_share_no_memory_with_pending_work(nats):
    """A block freed while the current stream still has a write to it under way is not handed to a call on another
    stream; nor is what such a call returned, freed while the current stream still reads it, handed out again."""
    rng = torch.Generator().manual_seed(15)
    table, _, k, v = _filled(rng, [300], 16, 2, 128, BF)
    c = _cache(nats, table, [300], k, v)
    q = torch.randn(1, 8, 128, generator=rng).to(BF).cuda()
    f = nats.rope_inv_freq(128)
    x = torch.randn(1, 8, 64, 128, generator=rng).to(BF).cuda()
    n_new = torch.tensor([1], dtype=torch.int32).cuda()
    kv = torch.zeros(1, 2, 64, 128, dtype=BF, device="cuda")
    start = torch.tensor([0], dtype=torch.int32).cuda()
    c2 = nats.PagedCache.empty(4, 16, 2, 128, 1, 4)
    c2.table.copy_(torch.arange(4, dtype=torch.int32)[None])
    calls = [lambda s: nats.paged_decode(c, q, stream=s), lambda s: nats.qk_norm_rope(x, x, None, None, f, stream=s)[0],
             lambda s: nats.paged_append(c2, kv, kv, start=start, n_new=n_new, q=x, stream=s)]
    want = [call(None) for call in calls]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call, w in zip(calls, want):
        for _ in range(3):
            torch.cuda._sleep(20_000_000)  # about 10 ms
            for _ in range(8):
                torch.empty_like(w).fill_(7)  # freed with its write still to run
            got = call(s)
            s.synchronize()
            assert torch.equal(got.cpu(), w.cpu())
            torch.cuda.synchronize()
            assert torch.equal(got, w)
            with torch.cuda.stream(s):
                keep = got.clone()
            s.synchronize()
            torch.cuda._sleep(20_000_000)
            late = got * 1  # the current stream reads it late
            del got
            others = [call(s).fill_(9) for _ in range(4)]
            torch.cuda.synchronize()
            assert torch.equal(late, keep)
            del others


# ------------------------------------------------------------------ append

APPEND = [
    # T, n_new, start, Hq, Hk, d, page, dtype, norm, rot, interleaved
    (1, None, [5, 0, 31], 4, 2, 64, 16, BF, True, 64, False),
    (40, [40, 0, 13], [0, 9, 20], 6, 2, 128, 16, BF, True, 128, False),
    (33, [33, 1, 32], [15, 16, 17], 3, 3, 64, 48, F32, True, 32, True),
    (7, None, [3, 60, 64], 0, 1, 128, 64, BF, True, 112, False),
    (21, [5, 21, 0], None, 2, 1, 64, 32, F32, False, 64, False),
    (130, [100, 130, 64], [1, 2, 3], 4, 4, 128, 128, BF, False, 0, False),
]


@pytest.mark.parametrize("T,n_new,start,Hq,Hk,d,page,dtype,norm,rot,inter", APPEND)
def test_append(nats, T, n_new, start, Hq, Hk, d, page, dtype, norm, rot, inter):
    B = 3
    rng = torch.Generator().manual_seed(T)
    lens = [11, 0, 30]
    first = lens if start is None else start
    table, _, n_pages = ref.assign([p + T for p in first], page, rng, 2)
    k0 = torch.randn(n_pages, Hk, page, d, generator=rng).to(dtype)
    v0 = torch.randn(n_pages, Hk, page, d, generator=rng).to(dtype)
    w0 = torch.rand(n_pages, Hk, page, generator=rng)
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=rng).to(dtype)
    split = lambda t: [t[..., a * d:b * d].unflatten(-1, (b - a, d)).transpose(1, 2)
                       for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk))]
    q, k, v = split(qkv)
    gq, gk, gv = split(qkv.cuda())
    wq, wk = 1 + 0.3 * torch.randn(d, generator=rng), 1 + 0.3 * torch.randn(d, generator=rng)
    f = torch.tensor([1e6 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64) if rot else None
    c = _cache(nats, table, lens, k0, v0, w0)
    out_q = torch.full((B, Hq, T, d), 9.0, dtype=dtype, device="cuda") if Hq else None
    dev = lambda x, dt=torch.int32: None if x is None else torch.tensor(x, dtype=dt).cuda()
    r = nats.paged_append(c, gk, gv, start=dev(start), n_new=dev(n_new), q=gq if Hq else None, out_q=out_q, norm=norm,
                          w_q=wq.cuda(), w_k=wk.cuda(), inv_freq=None if f is None else f.cuda(), interleaved=inter)
    assert r is out_q
    c.check()
    counts = [T] * B if n_new is None else n_new
    pos = torch.tensor(first)[:, None] + torch.arange(T)
    kr, kz = ref.norm_rotate(k, wk, pos, f, inter, norm, 1e-6), ref.norm_rotate(k, wk, pos, None, inter, norm, 1e-6)
    kb = ref.rope_bound(kr, kz, rot, inter, dtype)
    gotk, gotv, gotw = c.k_pages.cpu(), c.v_pages.cpu(), c.weight.cpu()
    untouched = torch.ones(n_pages, page, dtype=torch.bool)
    for b in range(B):
        j = first[b] + torch.arange(counts[b])
        at, sl = table[b].long()[j // page], j % page
        untouched[at, sl] = False
        n = counts[b]
        assert ((gotk[at, :, sl].transpose(0, 1).double() - kr[b, :, :n]).abs() <= kb[b, :, :n]).all()
        assert torch.equal(gotv[at, :, sl].transpose(0, 1), v[b, :, :n])
        assert (gotw[at, :, sl] == 0).all()
    for got, was in ((gotk, k0), (gotv, v0), (gotw, w0)):
        assert torch.equal(got.transpose(1, 2)[untouched], was.transpose(1, 2)[untouched])
    if Hq:
        qr, qz = ref.norm_rotate(q, wq, pos, f, inter, norm, 1e-6), ref.norm_rotate(q, wq, pos, None, inter, norm, 1e-6)
        qb = ref.rope_bound(qr, qz, rot, inter, dtype)
        for b in range(B):
            n = counts[b]
            assert ((out_q[b, :, :n].cpu().double() - qr[b, :, :n]).abs() <= qb[b, :, :n]).all()
            assert (out_q[b, :, n:] == 9).all()


# more tokens than warps run at once, few rows each: a group of lanes takes a token of its own
@pytest.mark.parametrize("T,n_new,start,Hq,Hk,d,page,dtype,norm,rot,inter", [
    (1301, [1301, 0, 777], [5, 0, 31], 4, 2, 128, 16, BF, True, 128, False),
    (1301, None, None, 1, 3, 64, 48, F32, True, 32, True),
])
def test_append_of_many_tokens(nats, T, n_new, start, Hq, Hk, d, page, dtype, norm, rot, inter):
    test_append(nats, T, n_new, start, Hq, Hk, d, page, dtype, norm, rot, inter)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_append_of_many_tokens_outside_the_table_or_pool(nats, dtype, d):
    """One call writes what calls of so few tokens write that the rows of one lie side by side, and reports the same."""
    rng = torch.Generator().manual_seed(19)
    B, T, page, Hk, Hq = 3, 1301, 16, 2, 1
    table, _, n_pages = ref.assign([T, T, T], page, rng, 2)
    table[1, 40], table[2, 5:] = n_pages, -1
    table = table[:, :75]  # the last 101 tokens of each lie outside
    start, n_new = torch.tensor([0, 3, 0], dtype=torch.int32), torch.tensor([1301, 1200, 1], dtype=torch.int32)
    x = [torch.randn(B, h, T, d, generator=rng).to(dtype).cuda() for h in (Hq, Hk, Hk)]
    f = nats.rope_inv_freq(d)
    pools = []
    for step in (T, 400):
        w = torch.ones(n_pages, Hk, page)
        c = _cache(nats, table, [0] * B, *_pool(rng, n_pages, Hk, page, d, dtype, garbage=False), w)
        out = torch.full_like(x[0], 5.0)
        for a in range(0, T, step):
            q, k, v = (y[:, :, a:a + step] for y in x)
            nats.paged_append(c, k, v, start=(start + a).cuda(), n_new=(n_new - a).clamp(min=0).cuda(), q=q,
                              out_q=out[:, :, a:a + step], norm=True, inv_freq=f)
        with pytest.raises(nats.NatsError):
            c.check()
        pools.append([c.k_pages, c.v_pages, c.weight, out])
    for one, parts in zip(*pools):
        assert torch.equal(one, parts)
    assert (pools[0][3][2, :, 1:] == 5).all() and not (pools[0][3][0] == 5).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_from_odd_addresses(nats, dtype):
    """Rows that start at odd entries move entry by entry, to the same values."""
    rng = torch.Generator().manual_seed(14)
    T, Hq, Hk, d = 9, 3, 2, 64
    buf = torch.randn(2, T, (Hq + 2 * Hk) * d + 3, generator=rng).to(dtype).cuda()
    parts = [buf[..., 1 + a * d:1 + b * d].unflatten(-1, (b - a, d)).transpose(1, 2) for a, b in ((0, 3), (3, 5), (5, 7))]
    f = nats.rope_inv_freq(64)
    res = []
    for q, k, v in (parts, [p.contiguous() for p in parts]):
        c = nats.PagedCache.empty(4, 16, Hk, d, 2, 2, dtype=dtype)
        c.table.copy_(torch.tensor([[3, 1], [0, 2]], dtype=torch.int32))
        q = nats.paged_append(c, k, v, q=q, norm=True, inv_freq=f, start=torch.tensor([10, 0], dtype=torch.int32).cuda())
        res.append((q, c.k_pages, c.v_pages))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    assert torch.equal(res[0][2][0, :, :9], parts[2][1])


def test_append_given_positions_and_new_query(nats):
    rng = torch.Generator().manual_seed(9)
    c = nats.PagedCache.empty(4, 16, 1, 64, 2, 2, dtype=F32)
    c.table.copy_(torch.tensor([[3, 1], [0, 2]], dtype=torch.int32))
    x = torch.randn(2, 1, 5, 64, generator=rng).cuda()
    pos = torch.tensor([[7, 900, 3, 2, 1], [5, 5, 5, 5, 5]]).cuda()
    f = nats.rope_inv_freq(64)
    oq = nats.paged_append(c, x, x, q=x, norm=True, inv_freq=f, positions=pos,
                           n_new=torch.tensor([5, 2], dtype=torch.int32).cuda())
    want, _ = nats.qk_norm_rope(x, x, None, None, f, pos)
    assert torch.equal(oq[0], want[0]) and torch.equal(oq[1, :, :2], want[1, :, :2]) and (oq[1, :, 2:] == 0).all()
    assert torch.equal(c.k_pages[3, 0, :5], want[0, 0]) and torch.equal(c.k_pages[0, 0, :2], want[1, 0, :2])
    assert (c.k_pages[0, 0, 2:] == 0).all() and (c.lens == 0).all()


def test_append_outside_the_table_or_pool(nats):
    """Tokens behind the table, before slot 0 or on a page that is not the pool's are left out and reported; the
    others, and the queries, are written."""
    c = nats.PagedCache.empty(3, 16, 2, 64, 3, 2, dtype=BF)
    c.table.copy_(torch.tensor([[1, -1], [0, 2], [99, 0]], dtype=torch.int32))
    x = torch.ones(3, 2, 4, 64, dtype=BF, device="cuda")
    start = torch.tensor([14, 30, -2], dtype=torch.int32).cuda()
    oq = nats.paged_append(c, x, 2 * x, start=start, q=x)
    assert (oq == 1).all()
    k = c.k_pages[:, 0, :, 0].cpu()
    want = torch.zeros(3, 16)
    want[1, 14:] = 1  # sequence 0: slots 14, 15; 16, 17 have no page
    want[2, 14:] = 1  # sequence 1: slots 30, 31; 32, 33 lie behind the table
    assert torch.equal(k.float(), want) and torch.equal(c.v_pages[:, 1, :, 3].cpu().float(), 2 * want)
    with pytest.raises(nats.NatsError):
        c.check()


def test_append_captured_follows_the_lengths(nats):
    c = nats.PagedCache.empty(4, 16, 1, 64, 1, 4, dtype=BF)
    c.table.copy_(torch.arange(4, dtype=torch.int32)[None])
    x = torch.zeros(1, 1, 1, 64, dtype=BF, device="cuda")
    nats.paged_append(c, x, x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nats.paged_append(c, x, x)
        c.lens.add_(1)
    for i in range(40):
        x.fill_(i + 1)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.k_pages[:, 0, :, 0].reshape(-1).cpu().float(),
                       torch.cat([torch.arange(1, 41), torch.zeros(24, dtype=torch.int64)]).float())
    assert int(c.lens) == 40


# ------------------------------------------------------------------- evict

EVICT = [
    # lens, Hk, d, page, dtype, budget, recent, sinks, weights
    ([100], 1, 64, 16, BF, 40, 0, 0, "spread"),
    ([100, 39, 40, 41, 0, 1], 2, 64, 16, F32, 40, 10, 2, "spread"),
    ([2112, 1500], 3, 128, 64, BF, 1000, 256, 4, "spread"),
    ([500, 300], 2, 128, 48, BF, 128, 0, 4, "ties"),
    ([500], 2, 64, 32, F32, 65, 64, 1, "ties"),
    ([500], 1, 64, 16, BF, 33, 20, 13, "spread"),
    ([300, 200], 2, 64, 128, BF, 100, 3, 1, "odd"),
    ([5000], 1, 64, 16, F32, 4097, 1, 0, "equal"),
    ([30000, 1025], 1, 64, 64, BF, 1025, 100, 4, "spread"),
    ([64, 10], 1, 64, 16, BF, 0, 0, 0, "spread"),
    ([500, 450, 301], 2, 128, 32, F32, 300, 20, 4, "odd"),
    ([512, 513, 511], 2, 64, 64, BF, 200, 10, 2, "odd"),
    ([5000, 600], 1, 64, 16, BF, 200, 10, 2, "odd"),
    ([5000, 600], 1, 128, 16, F32, 600, 0, 600, "odd"),
]


@pytest.mark.parametrize("lens,Hk,d,page,dtype,budget,recent,sinks,kind", EVICT)
def test_evict(nats, lens, Hk, d, page, dtype, budget, recent, sinks, kind):
    rng = torch.Generator().manual_seed(budget + len(lens))
    per = -(-budget // page) + 1
    table, spare, k, v = _filled(rng, lens, page, Hk, d, dtype, extra=per * len(lens) + 1)
    shape = k.shape[:3]
    w = {"spread": torch.exp(3 * torch.randn(shape, generator=rng)),
         "ties": torch.randint(0, 4, shape, generator=rng).float(),
         "equal": torch.full(shape, 2.5),
         "odd": torch.randint(-3, 3, shape, generator=rng).float()}[kind]
    if kind == "odd":  # the values that order strangely: both zeros, infinities, NaN, the lowest and the smallest
        strange = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, -math.nan, 1e-45, -1e-45, -3.4e38])
        w = strange[torch.randint(0, 9, shape, generator=rng)]
    out_table = spare[:per * len(lens)].reshape(len(lens), per).clone()
    c = _cache(nats, table, lens, k, v, w)
    keep, n = nats.paged_evict(c, out_table.cuda(), budget, recent=recent, sinks=sinks, return_keep=True)
    c.check()
    want = ref.evict(w, table, lens, page, budget, recent, sinks)
    assert torch.equal(keep.cpu(), want)
    assert n.cpu().tolist() == [min(x, budget) for x in lens] and c.lens.cpu().tolist() == lens
    gk, gv, gw = c.k_pages.cpu(), c.v_pages.cpu(), c.weight.cpu()
    ints = {BF: torch.int16, F32: torch.int32}[dtype]
    touched = torch.zeros(shape[0], page, dtype=torch.bool)
    for b, m in enumerate(n.cpu().tolist()):
        i = torch.arange(m)
        at, sl = out_table[b].long()[i // page], i % page
        touched[at, sl] = True
        for h in range(Hk):
            src = want[b, h, :m].long()
            fr = (table[b].long()[src // page], h, src % page)
            assert torch.equal(gk[at, h, sl].view(ints), k[fr].view(ints))
            assert torch.equal(gv[at, h, sl].view(ints), v[fr].view(ints))
            assert torch.equal(gw[at, h, sl].view(torch.int32), w[fr].view(torch.int32))
    for got, was in ((gk, k), (gv, v)):
        assert torch.equal(got.transpose(1, 2)[~touched].view(ints), was.transpose(1, 2)[~touched].view(ints))
    assert torch.equal(gw.transpose(1, 2)[~touched].view(torch.int32), w.transpose(1, 2)[~touched].view(torch.int32))


@pytest.mark.parametrize("max_pages", [1024, 2048])  # clusters of eight CTAs of 512 and of 1024 threads
@pytest.mark.parametrize("lens", [[300, 50], [512, 511], [513, 1], [1024, 1025], [101, 2048]])
def test_evict_short_sequences_in_long_tables(nats, max_pages, lens):
    rng = torch.Generator().manual_seed(max_pages + lens[0])
    page, budget = 64, 100
    table, spare, k, v = _filled(rng, lens, page, 2, 64, BF, extra=2 * len(lens))
    w = torch.rand(k.shape[:3], generator=rng)
    wide = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    c = _cache(nats, wide, lens, k, v, w)
    # what the kernels before left in shared memory must not matter: one of them ran on full sequences
    long = nats.PagedCache(c.k_pages, c.v_pages, torch.full((1, max_pages), int(table[0, 0]), dtype=torch.int32).cuda(),
                           torch.tensor([max_pages * page], dtype=torch.int32).cuda(), weight=c.weight)
    nats.paged_evict(long, spare[None, :2].cuda(), budget)
    c.k_pages.copy_(k), c.v_pages.copy_(v), c.weight.copy_(w)
    keep, n = nats.paged_evict(c, spare.reshape(len(lens), 2).cuda(), budget, recent=7, sinks=3, return_keep=True)
    c.check()
    assert torch.equal(keep.cpu(), ref.evict(w, wide, lens, page, budget, 7, 3))
    assert n.cpu().tolist() == [min(x, budget) for x in lens]


def test_evict_of_many_heads(nats):
    """More heads than two to an SM: each is copied by the CTA that selects it."""
    test_evict(nats, [600 - 13 * b for b in range(20)], 16, 64, 16, F32, 400, 30, 2, "ties")


def test_evict_bad_entries_are_reported(nats):
    rng = torch.Generator().manual_seed(10)
    table, spare, k, v = _filled(rng, [64], 16, 1, 64, F32, extra=2)
    w = torch.rand(k.shape[:3], generator=rng)
    bad = table.clone()
    bad[0, 1] = -1  # its slots count as the lowest weight
    c = _cache(nats, bad, [64], k, v, w)
    keep, _ = nats.paged_evict(c, spare[None].cuda(), 32, return_keep=True)
    assert not ((keep >= 16) & (keep < 32)).any()
    c.check()  # none of them is copied
    c2 = _cache(nats, table, [64], k, v, w)
    nats.paged_evict(c2, torch.tensor([[int(spare[0]), 1 << 20]], dtype=torch.int32).cuda(), 32)
    with pytest.raises(nats.NatsError):
        c2.check()


def test_every_operator_captured_behind_copies_and_forks(nats):
    """A graph in which each operator's kernels follow a memory copy, a fill, another stream's work and each other."""
    rng = torch.Generator().manual_seed(16)
    table, spare, k, v = _filled(rng, [200, 90], 16, 2, 64, BF, extra=8)
    c = _cache(nats, table, [200, 90], k, v, torch.zeros(k.shape[:3]))
    ot = spare.reshape(2, 4).contiguous().cuda()
    f, n = nats.rope_inv_freq(64), torch.tensor([200, 90], dtype=torch.int32).cuda()
    host = torch.randn(2, 6, 1, 64, generator=rng).to(BF).pin_memory()
    x, kv = torch.empty(2, 6, 1, 64, dtype=BF, device="cuda"), torch.randn(2, 2, 1, 64, generator=rng).to(BF).cuda()
    start = n - 1

    def steps(side):
        x.copy_(host, non_blocking=True)
        q = nats.paged_append(c, kv, kv, start=start, q=x, norm=True, inv_freq=f)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            r = nats.qk_norm_rope(x, x, None, None, f)
            g = nats.qk_norm_rope_bwd(*r, x, x, None, None, f)
        c.weight.zero_()
        out = nats.paged_decode(c, q[:, :, 0], accumulate=True)
        torch.cuda.current_stream().wait_stream(side)
        keep, m = nats.paged_evict(c, ot, 60, recent=5, return_keep=True)
        return [q, out, r[0], g["dq"], g["dw_q"], c.weight, keep, m]

    want = [t.clone() for t in steps(torch.cuda.Stream())]
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(side)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_evict_captured(nats):
    rng = torch.Generator().manual_seed(11)
    table, spare, k, v = _filled(rng, [200, 90], 16, 2, 64, BF, extra=8)
    w = torch.rand(k.shape[:3], generator=rng)
    c = _cache(nats, table, [200, 90], k, v, w)
    ot = spare.reshape(2, 4).contiguous().cuda()
    nats.paged_evict(c, ot, 60)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        keep, n = nats.paged_evict(c, ot, 60, recent=5, return_keep=True)
    w2 = torch.rand(k.shape[:3], generator=rng)
    c.weight.copy_(w2)
    c.lens.copy_(torch.tensor([100, 50], dtype=torch.int32))
    g.replay()
    assert torch.equal(keep.cpu(), ref.evict(w2, table, [100, 50], 16, 60, 5, 0)) and n.tolist() == [60, 50]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,Hq,Hk,d,page", [(BF, 8, 2, 64, 16), (F32, 4, 4, 128, 32), (BF, 6, 1, 128, 64)])
def test_prompt_steps_and_eviction_together(nats, dtype, Hq, Hk, d, page):
    """A ragged prompt, decode steps that sum weights, an eviction, more steps: each step's output against the 64-bit
    attention over what the cache holds, the kept slots against the sort of the cache's own weights, and every key
    against its own norm and rotation in 64 bits."""
    B, budget, recent, sinks = 3, 96, 24, 2
    rng = torch.Generator().manual_seed(12)
    prompt = [150, 40, 97]
    most = 20
    n_pages = 3 * B * most
    c = nats.PagedCache.empty(n_pages, page, Hk, d, B, most, dtype=dtype, weight=True)
    pages = torch.randperm(n_pages, generator=rng).to(torch.int32)
    c.table.copy_(pages[:B * most].reshape(B, most))
    fresh = pages[B * most:2 * B * most].reshape(B, most).contiguous().cuda()
    f = nats.rope_inv_freq(d, 1e6)
    wq, wk = torch.full((d,), 1.5, device="cuda"), torch.full((d,), 1.2, device="cuda")
    seen = torch.zeros(B, dtype=torch.int32, device="cuda")  # tokens so far: the rotation's positions

    def tokens(T, n_new):
        qkv = torch.randn(B, T, (Hq + 2 * Hk) * d, generator=rng).to(dtype).cuda()
        q, k, v = (t.unflatten(-1, (-1, d)).transpose(1, 2) for t in qkv.split([Hq * d, Hk * d, Hk * d], -1))
        pos = seen[:, None].long() + torch.arange(T, device="cuda")
        at = c.lens.clone()
        oq = nats.paged_append(c, k, v, n_new=n_new, q=q, norm=True, w_q=wq, w_k=wk, inv_freq=f, positions=pos)
        kr = ref.norm_rotate(k.cpu(), wk.cpu(), pos.cpu(), f.cpu(), False, True, 1e-6)
        kz = ref.norm_rotate(k.cpu(), wk.cpu(), pos.cpu(), None, False, True, 1e-6)
        bound = ref.rope_bound(kr, kz, d, False, dtype)
        c.lens.add_(n_new)
        seen.add_(n_new)
        pool = c.k_pages.cpu()
        for b in range(B):
            m = int(n_new[b])
            got = ref.slots(pool, c.table.cpu(), b, int(c.lens[b]), page)[:, int(at[b]):]
            assert ((got.double() - kr[b, :, :m]).abs() <= bound[b, :, :m]).all()
        return oq

    def step():
        q = tokens(1, torch.ones(B, dtype=torch.int32, device="cuda"))[:, :, 0]
        before = c.weight.double().sum()
        out = nats.paged_decode(c, q, accumulate=True)
        e, _, _, err, _ = ref.decode(q.cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu(), c.lens.tolist())
        assert ((out.cpu().double() - e).abs() <= ref.HALF[dtype] * (e.abs() + err) + err).all()
        assert abs(float(c.weight.double().sum() - before) - B * Hq) < 1e-3 * Hq

    tokens(150, torch.tensor(prompt, dtype=torch.int32, device="cuda"))
    for _ in range(3):
        step()
    lens = c.lens.tolist()
    keep, n = nats.paged_evict(c, fresh, budget, recent=recent, sinks=sinks, return_keep=True)
    assert torch.equal(keep.cpu(), ref.evict(c.weight.cpu(), c.table.cpu(), lens, page, budget, recent, sinks))
    c.table.copy_(fresh)
    c.lens.copy_(n)
    for _ in range(3):
        step()
    c.check()
    assert c.lens.tolist() == [min(x, budget) + 3 for x in lens] and seen.tolist() == [p + 6 for p in prompt]


def test_refusals(nats):
    c = nats.PagedCache.empty(4, 16, 2, 64, 2, 2, dtype=BF)
    cw = nats.PagedCache.empty(4, 16, 2, 64, 2, 2, dtype=BF, weight=True)
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    k = torch.zeros(2, 2, 1, 64, dtype=BF, device="cuda")
    ot = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        nats.paged_decode(c, q, accumulate=True)  # no weights
    with pytest.raises(ValueError):
        nats.paged_evict(c, ot, 8)
    with pytest.raises(ValueError):
        nats.paged_decode(c, q[:1])
    with pytest.raises(TypeError):
        nats.paged_decode(c, q.float())
    with pytest.raises(nats.NatsError):
        nats.paged_decode(c, q[:, :3])  # not a multiple of the key heads
    with pytest.raises(nats.NatsError):
        nats.paged_decode(c, q, scale=float("nan"))
    with pytest.raises(nats.NatsError):
        nats.paged_decode(c, q, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        nats.paged_append(c, k[:, :1], k[:, :1])
    with pytest.raises(TypeError):
        nats.paged_append(c, k, k, start=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(nats.NatsError):
        nats.paged_evict(cw, ot, 8, recent=6, sinks=3)
    with pytest.raises(nats.NatsError):
        nats.paged_evict(cw, ot, 33)  # two pages hold 32
    with pytest.raises(nats.NatsError):
        nats.paged_evict(cw, cw.table, 8)
    with pytest.raises(ValueError):
        nats.paged_evict(cw, ot, (1 << 32) + 8)
    with pytest.raises(nats.NatsError):
        nats.paged_evict(cw, ot, 8, lens_out=cw.lens)
    with pytest.raises(ValueError):
        nats.PagedCache(c.k_pages, c.v_pages[:2], c.table, c.lens)
    with pytest.raises(TypeError):
        nats.PagedCache(c.k_pages, c.v_pages, c.table.long(), c.lens)
    with pytest.raises(AttributeError):
        c.table = c.table.clone()


@pytest.mark.parametrize("B,Hk,n,page,budget,recent,sinks", [
    (1, 1, 300000, 64, 70000, 100, 4), (1, 2, 1000000, 64, 3, 1, 1), (2, 30, 40000, 16, 39000, 0, 0),
    (1, 200, 9000, 48, 100, 7, 0)])
def test_evict_long_sequences(nats, B, Hk, n, page, budget, recent, sinks):
    """Heads of several CTAs, and shares longer than a CTA holds: the kept slots of a stable sort."""
    torch.manual_seed(n)
    pg, per = -(-n // page), -(-budget // page)
    N = B * (pg + per)
    k = torch.zeros(N, Hk, page, 64, dtype=BF, device="cuda")
    w = 3 * torch.randn(N, Hk, page, device="cuda")
    if n % 20000 == 0:  # with many ties
        w = w.round() / 3
    order = torch.randperm(N, device="cuda").int()
    table, ot = order[:B * pg].reshape(B, pg).contiguous(), order[B * pg:].reshape(B, per).contiguous()
    lens = torch.tensor([n - 3 * b for b in range(B)], dtype=torch.int32, device="cuda")
    c = nats.PagedCache(k, k.clone(), table, lens, weight=w)
    ww = w[table.long()].transpose(1, 2).reshape(B, Hk, -1)[:, :, :n].clone()
    j, L = torch.arange(n, device="cuda"), lens.long()[:, None, None]
    key = torch.where((j < sinks) | (j >= L - recent), math.inf, ww)
    key = torch.where(j < L, key, -math.inf)
    want = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget].sort(dim=-1).values.int()
    keep, _ = nats.paged_evict(c, ot, budget, recent=recent, sinks=sinks, return_keep=True)
    assert torch.equal(keep, want)
