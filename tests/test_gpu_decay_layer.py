"""Layer norm and linear attention with a decay together, as a layer uses them:
norm, projection, attention, norm of each head's output, projection; its
training step against a 64-bit one, and a prompt that goes on token by token."""

import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

B, L, H, d, hidden = 2, 200, 4, 64, 256


@pytest.fixture(scope="module")
def nats():
    import linear_attention_nats_gb300 as n

    return n


def inputs():
    gen = torch.Generator().manual_seed(3)
    z = lambda *s, std=1.0: torch.randn(*s, generator=gen, dtype=torch.float64) * std
    p = dict(x=z(B, L, hidden) + 0.5, w1=1 + z(hidden, std=0.1), b1=z(hidden, std=0.1), wi=z(hidden, 3 * H * d, std=hidden ** -0.5),
             w2=1 + z(d, std=0.1), b2=z(d, std=0.1), wo=z(H * d, hidden, std=(H * d) ** -0.5), dy=z(B, L, hidden))
    g = torch.tensor([-0.5, -0.1, -0.02, -0.001])
    return {n: t.float() for n, t in p.items()}, g


def wanted(p, g):
    """The layer in 64 bits from its definition, gradients by autograd."""
    p = {n: t.double() for n, t in p.items()}
    for n in p:
        p[n].requires_grad_(n != "dy")

    def norm(x, w, b):
        c = x - x.mean(-1, keepdim=True)
        return c / (c.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w + b

    qkv = (norm(p["x"], p["w1"], p["b1"]) @ p["wi"]).view(B, L, 3, H, d)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    i = torch.arange(L)
    D = torch.where(i[:, None] >= i, torch.exp(g.double()[:, None, None] * (i[:, None] - i).clamp(min=0)), 0.0)
    o = (q @ k.mT * D) @ v * d ** -0.5
    y = norm(o, p["w2"], p["b2"]).transpose(1, 2).reshape(B, L, H * d) @ p["wo"]
    (y * p["dy"]).sum().backward()
    return y.detach(), {n: t.grad for n, t in p.items() if n != "dy"}


def close(got, want, what):
    """Each of five stages rounds by at most (d + 200) 2 U of its terms' magnitudes, which are below 10 times the
    results' largest here: 5 * 10 * 2 * 264 * 2^-24 = 1.6e-3."""
    e = float((got.cpu().double() - want).abs().max() / want.abs().max())
    assert e < 1.6e-3, (what, e)


def test_training_step(nats):
    p, g = inputs()
    want, grads = wanted(p, g)
    c = {n: t.cuda() for n, t in p.items()}
    g = g.cuda()
    z = nats.layer_norm(c["x"], c["w1"], c["b1"])
    qkv = (z @ c["wi"]).view(B, L, 3, H, d)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    o = nats.decay_attn(q, k, v, g)
    # each head's norm, straight into the layout of the output projection
    h = torch.empty(B, L, H, d, device="cuda")
    nats.layer_norm(o, c["w2"], c["b2"], out=h.transpose(1, 2))
    y = h.view(B, L, H * d) @ c["wo"]
    close(y, want, "y")
    # back
    dh = (c["dy"] @ c["wo"].T).view(B, L, H, d)
    close(h.view(-1, H * d).T @ c["dy"].view(-1, hidden), grads["wo"], "wo")
    r2 = nats.layer_norm_bwd(dh.transpose(1, 2), o, c["w2"])
    dqkv = torch.empty_like(qkv)
    nats.decay_attn_bwd(r2["dx"], q, k, v, g, **{n: dqkv[:, :, i].transpose(1, 2) for i, n in enumerate(("dq", "dk", "dv"))})
    dqkv = dqkv.view(B * L, 3 * H * d)
    close(z.view(-1, hidden).T @ dqkv, grads["wi"], "wi")
    r1 = nats.layer_norm_bwd((dqkv @ c["wi"].T).view(B, L, hidden), c["x"], c["w1"])
    for n, t in (("x", r1["dx"]), ("w1", r1["dw"]), ("b1", r1["db"]), ("w2", r2["dw"]), ("b2", r2["db"])):
        close(t, grads[n], n)
    nats.decay_attn_check()


def test_prompt_and_tokens(nats):
    """The layer over a padded batch of prompts and then token by token: the rows of the whole prompt."""
    p, g = inputs()
    want, _ = wanted(p, g)
    c = {n: t.cuda() for n, t in p.items()}
    g = g.cuda()
    lens = [150, 90]

    def heads(x):
        qkv = (nats.layer_norm(x, c["w1"], c["b1"]) @ c["wi"]).view(*x.shape[:-1], 3, H, d)
        return [qkv[..., i, :, :] for i in range(3)]

    def tail(o):
        return nats.layer_norm(o, c["w2"], c["b2"]).reshape(*o.shape[:-2], H * d) @ c["wo"]

    q, k, v = (t.transpose(1, 2) for t in heads(c["x"]))
    o, state = nats.decay_attn(q, k, v, g, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), return_state=True)
    y = tail(o.transpose(1, 2))
    for b, n in enumerate(lens):
        close(y[b, :n], want[b, :n], ("prompt", b))
    for t in range(40):
        x = torch.stack([c["x"][b, n + t] for b, n in enumerate(lens)])
        y = tail(nats.decay_attn_step(*heads(x), g, state))
        close(y, torch.stack([want[b, n + t] for b, n in enumerate(lens)]), ("token", t))


def test_readme_layer(nats):
    """The README's lines as they stand there."""
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    lines = re.search(r"a prompt and then a token:\n\n((?:    .*\n)+)", text).group(1)
    p, _ = inputs()
    gen = torch.Generator().manual_seed(5)
    z = lambda *s: torch.randn(*s, generator=gen).cuda()
    tok = z(3, B, H, 128)
    env = dict(nats=nats, B=B, L=L, H=H, x=p["x"].cuda(), w=p["w1"].cuda(), b=p["b1"].cuda(), w_in=z(hidden, 3 * H * 128) / 16,
               log_decay=-torch.rand(H, generator=gen).cuda(), lens=torch.tensor([200, 130], dtype=torch.int32, device="cuda"),
               w_head=z(128), b_head=z(128), q1=tok[0], k1=tok[1], v1=tok[2])
    exec("\n".join(x[4:] for x in lines.splitlines()), env)
    o, state = nats.decay_attn(env["q"], env["k"], env["v"], env["log_decay"], lens=env["lens"], return_state=True)
    assert torch.equal(env["o"], nats.layer_norm(o, env["w_head"], env["b_head"]))
    a = torch.exp(env["log_decay"].double())[:, None, None]
    S = state.double() * a + tok[2].double()[..., None] * tok[1].double()[..., None, :]
    assert float((env["state"].double() - S).abs().max()) <= 4 * 2.0 ** -24 * float((state.abs().max() + 30))
    close(env["o1"], nats.layer_norm(((S @ tok[0].double()[..., None])[..., 0] * 128 ** -0.5).float(), env["w_head"],
                                     env["b_head"]).cpu().double(), "token")
