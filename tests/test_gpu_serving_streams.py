"""Calls on a stream other than the current one, whose arguments the caller frees as soon as they return."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def nats():
    from linear_attention_nats_gb300 import build

    build.build()
    import linear_attention_nats_gb300 as n

    return n


def _calls(nats):
    """name -> (arguments, call of them on a stream, what it gives)."""
    rng = torch.Generator().manual_seed(1)
    B, Hq, Hk, T, d, page, most = 2, 4, 2, 100, 64, 16, 8
    r = lambda *s: torch.randn(s, generator=rng).to(BF).cuda()
    table = torch.randperm(2 * B * most, generator=rng).int().cuda()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    n = 2 * B * most
    pool = dict(k_pages=r(n, Hk, page, d), v_pages=r(n, Hk, page, d), table=table[:B * most].view(B, most).clone(),
                lens=ints(100, 77), weight=torch.rand(n, Hk, page, generator=rng).cuda())
    q, k, f, pos = r(B, Hq, T, d), r(B, Hk, T, d), nats.rope_inv_freq(d), torch.arange(T, device="cuda")
    w = torch.rand(d, generator=rng).cuda()

    def rope(x, s):
        return nats.qk_norm_rope(x["q"], x["k"], x["w"], x["w2"], x["f"], x["pos"], stream=s)

    def back(x, s):
        g = nats.qk_norm_rope_bwd(x["gq"], x["gk"], x["q"], x["k"], x["w"], x["w2"], x["f"], x["pos"], stream=s)
        return tuple(g.values())

    def decode(x, s):
        c = nats.PagedCache(x["k_pages"], x["v_pages"], x["table"], x["lens"])
        return nats.paged_decode(c, x["q1"], return_lse=True, stream=s)

    def append(x, s):
        c = nats.PagedCache(x["k_pages"], x["v_pages"], x["table"], x["lens"], weight=x["weight"])
        return (nats.paged_append(c, x["k"], x["k2"], start=x["start"], n_new=x["n_new"], q=x["q"], norm=True, w_q=x["w"],
                                  inv_freq=x["f"], stream=s),)

    def evict(x, s):
        c = nats.PagedCache(x["k_pages"], x["v_pages"], x["table"], x["lens"], weight=x["weight"])
        return nats.paged_evict(c, x["out_table"], 40, recent=3, return_keep=True, stream=s)

    norm = dict(q=q, k=k, w=w, w2=w + 1, f=f, pos=pos)
    return {"rope": (norm, rope), "back": (dict(norm, gq=q + 1, gk=k - 1), back), "decode": (dict(pool, q1=r(B, Hq, d)), decode),
            "append": (dict(pool, k=k, k2=2 * k, q=q, w=w, f=f, start=ints(3, 9), n_new=ints(60, 100)), append),
            "evict": (dict(pool, out_table=table[B * most:].view(B, most).clone()), evict)}


@pytest.mark.parametrize("name", ["rope", "back", "decode", "append", "evict"])
def test_arguments_may_be_freed_before_a_call_on_another_stream_has_run(nats, name):
    args, call = _calls(nats)[name]
    copy = lambda: {n: t.clone() for n, t in args.items()}
    want = [t.clone() for t in call(copy(), None)]
    s = torch.cuda.Stream()
    for _ in range(3):
        mine = copy()
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(40_000_000)  # about 20 ms
        got = call(mine, s)
        del mine
        # what is allocated now takes up freed memory, and is written at once
        junk = [torch.empty_like(t).fill_(1) for _ in range(3) for t in args.values()]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk


@pytest.mark.parametrize("name", ["rope", "back", "decode", "append", "evict"])
def test_captured_on_a_forked_stream(nats, name):
    """A graph whose call runs on a second stream, with arguments made and freed inside the capture."""
    args, call = _calls(nats)[name]
    want = [t.clone() for t in call({n: t.clone() for n, t in args.items()}, None)]
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mine = {n: t.clone() for n, t in args.items()}
        side.wait_stream(torch.cuda.current_stream())
        got = call(mine, side)
        del mine
        torch.cuda.current_stream().wait_stream(side)
        out = [t.clone() for t in got]
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
