"""Outputs that share memory with an input of layer norm or of linear attention
with a decay: refused before anything runs where they may not, with every tensor
left as it was; in place where they may."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def refused(f, *tensors):
    before = [t.clone() for t in tensors]
    with pytest.raises(ValueError, match="share memory"):
        f()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, tensors))


def test_layer_norm(nats):
    buf = torch.randn(5, 64, device="cuda")
    x, u = buf[:4], torch.randn(4, 64, device="cuda")
    refused(lambda: nats.layer_norm(x, out=buf[1:]), buf)
    refused(lambda: nats.layer_norm_bwd(u, x, dx=buf[1:]), buf)
    refused(lambda: nats.layer_norm_bwd(x, u, dx=buf[1:]), buf)
    square = torch.randn(8, 8, 16, device="cuda")
    refused(lambda: nats.layer_norm(square, out=square.transpose(0, 1)), square)
    # the same rows, whatever the stride of a dimension of one
    one = torch.randn(3, 2, 64, device="cuda")
    want = nats.layer_norm(one[:1])
    nats.layer_norm(one[:1], out=one.as_strided((1, 2, 64), (7, 64, 1)))
    assert torch.equal(one[:1], want)
    # halves of one tensor's rows
    wide = torch.randn(6, 128, device="cuda")
    want = nats.layer_norm(wide[:, :64])
    nats.layer_norm(wide[:, :64], out=wide[:, 64:])
    assert torch.equal(wide[:, 64:], want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_decay_attn(nats, dtype):
    B, H, L, d = 2, 3, 40, 64
    q, k, v, u = (torch.randn(B, H, L, d, device="cuda").to(dtype) for _ in range(4))
    g = torch.full((H,), -0.1, device="cuda")
    for x in (q, k, v):
        refused(lambda: nats.decay_attn(q, k, v, g, out=x), q, k, v)
        refused(lambda: nats.decay_attn_bwd(u, q, k, v, g, dk=x), q, k, v, u)
    refused(lambda: nats.decay_attn_bwd(u, q, k, v, g, dv=u), q, k, v, u)
    one = torch.empty_like(q)
    refused(lambda: nats.decay_attn_bwd(u, q, k, v, g, dq=one, dv=one), one)
    long = torch.randn(B + 1, H, L, d, device="cuda").to(dtype)
    refused(lambda: nats.decay_attn(long[:B], k, v, g, out=long[1:]), long)
    qkv = torch.randn(B, L, 3, H, d, device="cuda").to(dtype)
    a = [qkv[:, :, i].transpose(1, 2) for i in range(3)]
    refused(lambda: nats.decay_attn(*a, g, out=a[1]), qkv)
    s = torch.randn(B + 1, H, d, d, device="cuda")
    refused(lambda: nats.decay_attn(q, k, v, g, state=s[:B], state_out=s[1:]), s)
    # inputs may be one another
    assert torch.equal(nats.decay_attn(q, q, q, g), nats.decay_attn(q, q.clone(), q.clone(), g))


def test_decay_attn_step(nats):
    q, k, v = (torch.randn(2, 3, 64, device="cuda") for _ in range(3))
    s, g = torch.randn(2, 3, 64, 64, device="cuda"), torch.full((3,), -0.1, device="cuda")
    for x in (q, k, v):
        refused(lambda: nats.decay_attn_step(q, k, v, g, s, out=x), q, k, v, s)
