"""Where linear attention with a decay cuts a sequence into segments: a call whose
heads fill the GPU walks it whole, and needs no workspace; with few heads it is
cut."""

import pytest
import torch

import decay_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def status(nats, x, g, out, bwd):
    """Of a call without a workspace: 1 (refused) where the sequence is cut."""
    B, H, L, d = x.shape
    n = nats._native
    dm = n.DecayDims(B, H, L, d, 0 if x.dtype == torch.bfloat16 else 1, 0.0)
    st = n.Strides(H * L * d, L * d, d)
    p = x.data_ptr()
    s = torch.cuda.current_stream().cuda_stream
    if bwd:
        return n.lib.nats_decay_attn_bwd(dm, p, st, p, st, p, st, p, st, g.data_ptr(), None, None, None, out[0].data_ptr(), st,
                                         out[1].data_ptr(), st, out[2].data_ptr(), st, None, None, 0, s)
    return n.lib.nats_decay_attn(dm, p, st, p, st, p, st, g.data_ptr(), None, None, out[0].data_ptr(), st, None, None, 0, s)


@pytest.mark.parametrize("H,L,d,dtype,bwd,cut", [
    (40, 4096, 128, torch.bfloat16, False, False), (64, 2048, 64, torch.bfloat16, False, False),
    (32, 2048, 128, torch.bfloat16, False, False), (160, 4096, 64, torch.bfloat16, False, False),
    (64, 8192, 64, torch.bfloat16, True, False), (512, 512, 128, torch.float32, False, False),
    (4, 8192, 128, torch.bfloat16, False, True), (16, 8192, 128, torch.bfloat16, False, True),
    (4, 4096, 64, torch.bfloat16, True, True), (4, 1024, 64, torch.float32, False, True)], ids=str)
def test_cut(nats, H, L, d, dtype, bwd, cut):
    x = torch.randn(1, H, L, d, device="cuda").to(dtype)
    out = [torch.empty_like(x) for _ in range(3)]
    assert status(nats, x, torch.full((H,), -0.1, device="cuda"), out, bwd) == (1 if cut else 0)
    torch.cuda.synchronize()


def test_few_segments(nats):
    """Many heads are cut into few parts."""
    f = nats._native.lib.nats_decay_attn_workspace_size
    assert f(nats._native.DecayDims(1, 100, 4096, 64, 1, 0.0)) <= 8 * 100 * 64 * 64 * 4
    assert f(nats._native.DecayDims(4, 16, 8192, 64, 1, 0.0)) <= 24 * 64 * 64 * 64 * 4


@pytest.mark.parametrize("H,L,d,bwd", [(64, 8192, 64, False), (8, 9000, 128, True)])
def test_values(nats, H, L, d, bwd):
    """At the cuts that are chosen, the first and last head against the 64-bit form."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    u, q, k, v = (torch.randn(1, H, L, d, generator=gen, device="cuda").bfloat16() for _ in range(4))
    g = torch.full((H,), -0.03, device="cuda")
    got = nats.decay_attn_bwd(u, q, k, v, g, state_grad=True) if bwd else nats.decay_attn(q, k, v, g, return_state=True)
    for h in (0, H - 1):
        c = [x[0, h:h + 1].cpu() for x in (u, q, k, v)]
        if bwd:
            rows = ref.attn_bwd(*c, g[:1].cpu(), d ** -0.5, L, None, None)
            for name, (x, size) in zip(("dq", "dk", "dv"), rows):
                e = (got[name][0, h].cpu().double() - x[0]).abs()
                assert (e <= ref.out_bound(x, size, d, L, torch.bfloat16, True)[0]).all(), name
            e = (got["dstate"][0, h].cpu().double() - rows[3][0][0]).abs()
            assert (e <= ref.state_bound(rows[3][1], L, False)[0]).all()
        else:
            o, size, S, S_size = ref.attn(*c[1:], g[:1].cpu(), d ** -0.5, L, None)
            e = (got[0][0, h].cpu().double() - o[0]).abs()
            assert (e <= ref.out_bound(o, size, d, L, torch.bfloat16, True)[0]).all()
            e = (got[1][0, h].cpu().double() - S[0]).abs()
            assert (e <= ref.state_bound(S_size, L, False)[0]).all()
