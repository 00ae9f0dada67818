"""A bounded wait that gives up inside the bf16 kernels of linear attention with
a decay: the kernels end, decay_attn_check reports it once, and the next call is
clean.  The wait is made to give up by nats_debug_decay_wait: one warp of each
CTA leaves its role at a given chunk, and the waits for its part run out."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def expire(nats, chunk):
    nats._native.lib.nats_debug_decay_wait(chunk)


def operands(B, H, L, d, lens):
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = [torch.randn(B, H, L, d, generator=gen, device="cuda").bfloat16() for _ in range(4)]
    g = -torch.rand(H, generator=gen, device="cuda")
    return x, g, torch.tensor(lens, dtype=torch.int32, device="cuda")


# three or four chunks, the last of them in time with tokens behind the end: the warp leaves two chunks ahead of that
# one, right ahead of it, at it, and (the last scan's order) behind it
@pytest.mark.parametrize("d,back,state,chunk", [(128, False, False, 1), (64, False, True, 1), (64, False, False, 2),
                                                (128, False, True, 0), (128, True, False, 0), (64, True, True, 1)])
def test_ragged(nats, d, back, state, chunk):
    (q, k, v, u), g, lens = operands(2, 4, 500, d, [500, 300])

    def call():
        if back:
            r = nats.decay_attn_bwd(u, q, k, v, g, lens=lens, state_grad=state)
            return [r[n] for n in sorted(r)]
        r = nats.decay_attn(q, k, v, g, lens=lens, return_state=state)
        return list(r) if state else [r]

    want = call()
    nats.decay_attn_check()
    expire(nats, chunk)
    call()
    with pytest.raises(nats.NatsError) as e:
        nats.decay_attn_check()
    assert e.value.code == 8
    nats.decay_attn_check()  # reported once
    again = call()
    nats.decay_attn_check()
    assert all(torch.equal(x, y) for x, y in zip(want, again))


def test_cut(nats):
    """In the kernels of a sequence cut into segments, those that form the states among them."""
    (q, k, v, u), g, lens = operands(2, 1, 9000, 128, [9000, 5000])
    assert nats._native.lib.nats_decay_attn_workspace_size(nats._native.DecayDims(2, 1, 9000, 128, 0, 0.0)) > 0
    want = nats.decay_attn(q, k, v, g, lens=lens, return_state=True)
    expire(nats, 0)
    nats.decay_attn(q, k, v, g, lens=lens, return_state=True)
    with pytest.raises(nats.NatsError):
        nats.decay_attn_check()
    again = nats.decay_attn(q, k, v, g, lens=lens, return_state=True)
    nats.decay_attn_check()
    assert all(torch.equal(x, y) for x, y in zip(want, again))


def test_cancelled(nats):
    (q, k, v, u), g, lens = operands(1, 2, 300, 64, [300])
    expire(nats, 0)
    expire(nats, -1)
    nats.decay_attn(q, k, v, g)
    nats.decay_attn_check()


def test_check_on_a_stream(nats):
    """The report is of the given stream's device, after the work on it."""
    (q, k, v, u), g, lens = operands(2, 4, 500, 128, [500, 300])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    expire(nats, 1)
    nats.decay_attn(q, k, v, g, lens=lens, stream=side)
    with pytest.raises(nats.NatsError):
        nats.decay_attn_check(side)
    nats.decay_attn_check(side)
