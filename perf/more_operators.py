"""Cases, plain forms and 64-bit values of layer norm (and its gradient) and of
linear attention with a decay for each head: over a prompt, its gradient, and
one new token on a kept state.

`own` chooses what `run` computes with: elementary torch operations in fp32,
or the library's operators.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64  # tokens of a chunk of the plain form


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's rows ahead of the layer's projection (hidden 2048): launch latency
        dict(name="norm tokens", op="norm", B=1, H=1, L=32, D=2048, type="bf16", layout="rows"),
        # the 1.3B-scale layer's input (B 4, L 8192, hidden 2048)
        dict(name="norm layer", op="norm", B=4, H=1, L=8192, D=2048, type="bf16", layout="rows"),
        # its training step, with the gradients of weight and bias
        dict(name="norm gradient", op="norm_grad", B=4, H=1, L=8192, D=2048, type="bf16", layout="rows"),
        # the norm of each head's output of an fp32 layer, its rows inside a [B, L, H, d] tensor
        dict(name="norm gradient heads", op="norm_grad", B=3, H=12, L=1021, D=64, type="f32", layout="heads"),
        # the layer's prefill (B 4, H 16, L 8192, d 128), q, k and v inside one projection's output
        dict(name="prompt", op="attn", B=4, H=16, L=8192, d=128, type="bf16", layout="packed", decay="slow", ragged=False,
             state=False),
        # a ragged batch of short prompts that go on from their states
        dict(name="prompt ragged", op="attn", B=9, H=16, L=1500, d=128, type="bf16", layout="heads", decay="fast", ragged=True,
             state=True),
        # one long document, few heads: the work has to be split over its length
        dict(name="prompt long", op="attn", B=1, H=8, L=131072, d=128, type="bf16", layout="heads", decay="slow", ragged=False,
             state=True),
        # an odd fp32 shape
        dict(name="prompt f32", op="attn", B=3, H=12, L=1021, d=64, type="f32", layout="packed", decay="slow", ragged=False,
             state=True),
        # the layer's training step
        dict(name="gradient", op="attn_grad", B=4, H=16, L=8192, d=128, type="bf16", layout="packed", decay="slow",
             ragged=False, state=False),
        # an fp32 one through a segment's state, padded to its longest sequence
        dict(name="gradient f32", op="attn_grad", B=2, H=12, L=1021, d=64, type="f32", layout="heads", decay="fast", ragged=True,
             state=True),
        # one new token of one sequence: launch latency
        dict(name="step", op="step", B=1, H=16, d=128, type="bf16", decay="slow"),
        # a serving batch's new tokens
        dict(name="step batch", op="step", B=96, H=16, d=128, type="bf16", decay="slow"),
    ]


MOST_BYTES = 1 << 29  # of a drawn case's pass; the largest listed one has about 2^30


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "attn", "attn", "attn", "attn_grad", "attn_grad", "step"])
        t = rng.choice(["bf16", "bf16", "bf16", "f32"])
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
        if op in ("norm", "norm_grad"):
            if rng.random() < 0.3:
                c = dict(op=op, B=_log(rng, 1, 16), H=H, L=_log(rng, 1, 8192), D=rng.choice([64, 128]), type=t,
                         layout=rng.choice(["heads", "rows"]))
            else:
                D = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 8, 1024), 128 * _log(rng, 1, 64)])
                c = dict(op=op, B=1, H=1, L=_log(rng, 1, 131072), D=D, type=t, layout="rows")
        elif op == "step":
            c = dict(op=op, B=_log(rng, 1, 256), H=H, d=rng.choice([64, 128, 128]), type=t,
                     decay=rng.choice(["slow", "fast"]))
        else:
            c = dict(op=op, B=_log(rng, 1, 32), H=H, L=_log(rng, 1, 65536), d=rng.choice([64, 128, 128]), type=t,
                     layout=rng.choice(["heads", "packed"]), decay=rng.choice(["slow", "fast"]),
                     ragged=rng.random() < 0.4, state=rng.random() < 0.5)
        if work(c)["bytes"] <= MOST_BYTES:
            return c


def _lens(c):
    """The batch's lengths: the padded length first, then shorter ones, an empty and a one-token sequence among them."""
    n, B = c["L"], c["B"]
    if not c["ragged"]:
        return [n] * B
    lens = [n - (n * 7 * b // (11 * B)) for b in range(B)]
    if B >= 8:
        lens[B // 2], lens[B // 3] = 0, 1
    return lens


def work(c):
    es = 2 if c["type"] == "bf16" else 4
    if c["op"] in ("norm", "norm_grad"):
        D, n = c["D"], c["B"] * c["H"] * c["L"] * c["D"]
        if c["op"] == "norm":
            return dict(bytes=2 * n * es + 8 * D, flops=8 * n)
        return dict(bytes=3 * n * es + 12 * D, flops=16 * n)
    d, BH = c["d"], c["B"] * c["H"]
    if c["op"] == "step":
        return dict(bytes=8 * BH * d * d + 4 * BH * d * es, flops=5 * BH * d * d)
    # a token: its outer product into the state, and the state's product with its query
    rows, out = sum(_lens(c)) * c["H"], BH * c["L"]
    state = 8 * BH * d * d if c["state"] else 0
    if c["op"] == "attn":
        return dict(bytes=(3 * rows + out) * d * es + state, flops=5 * rows * d * d)
    return dict(bytes=(4 * rows + 3 * out) * d * es + (12 * BH * d * d if c["state"] else 0), flops=12 * rows * d * d)


# ------------------------------------------------------------------ inputs

def _decays(c):
    """log decay of each head: reaches of 32 to 4096 tokens, or of one to 256."""
    h = torch.arange(c["H"], dtype=torch.float64)
    if c["decay"] == "slow":
        g = torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, c["H"] - 1)))
    else:
        g = -torch.exp2(-8.0 * (h + 1) / c["H"])
    return g.to(torch.float32).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c, dt = case, TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    s = dict(case=c)
    if c["op"] in ("norm", "norm_grad"):
        B, H, L, D = c["B"], c["H"], c["L"], c["D"]

        def rows():
            if c["layout"] == "heads":
                return normal(B, L, H, D).transpose(1, 2)
            return normal(B * H * L, D)

        x = rows()
        # rows of a residual stream: a mean and a spread of their own
        mean = torch.randn(x.shape[:-1] + (1,), generator=gen, device=DEV)
        spread = torch.exp(torch.randn(x.shape[:-1] + (1,), generator=gen, device=DEV))
        s["x"] = x.mul_(spread).add_(mean)
        s["w"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
        s["b"] = normal(D, std=0.1, dtype=torch.float32)
        if c["op"] == "norm_grad":
            s["dy"] = rows()
        return s
    B, H, d = c["B"], c["H"], c["d"]
    s["g"] = _decays(c)
    if c["op"] == "step":
        qkv = normal(B, 3, H, d)
        s["q"], s["k"], s["v"] = qkv[:, 0], qkv[:, 1], qkv[:, 2]
        s["state"] = normal(B, H, d, d, std=4.0, dtype=torch.float32)
        return s
    L = c["L"]
    if c["layout"] == "packed":
        qkv = normal(B, L, 3, H, d)
        s["q"], s["k"], s["v"] = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    else:
        s["q"], s["k"], s["v"] = (normal(B, H, L, d) for _ in range(3))
    s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV) if c["ragged"] else None
    s["state"] = normal(B, H, d, d, std=4.0, dtype=torch.float32) if c["state"] else None
    if c["op"] == "attn_grad":
        s["dout"] = normal(B, H, L, d)
        s["dstate"] = normal(B, H, d, d, dtype=torch.float32) if c["state"] else None
    return s


# -------------------------------------------------------------- plain forms

def _plain_norm(x, w, b):
    z = x.to(torch.float32)
    z = z - z.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)
    return (z * r * w + b).to(x.dtype)


def _plain_norm_grad(dy, x, w):
    z, u = x.to(torch.float32), dy.to(torch.float32)
    z = z - z.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)
    z = z * r
    lead = tuple(range(x.dim() - 1))
    t = u * w
    dx = r * (t - t.mean(-1, keepdim=True) - z * (t * z).mean(-1, keepdim=True))
    return dx.to(x.dtype), (u * z).sum(lead), u.sum(lead)


def _power(g, m):
    """g's decay over m tokens: [H, 1, 1, 1] and whole numbers [...] to [H, ...]; 1 at m = 0."""
    return torch.where(m == 0, 1.0, torch.exp(g * m.to(torch.float32)))


def _chunks(x, lens):
    """[B, H, L, d] in fp32 as [H, B, N, CHUNK, d], zero behind a sequence's end."""
    B, H, L, d = x.shape
    N = -(-L // CHUNK)
    y = torch.zeros((H, B, N * CHUNK, d), device=x.device)
    y[:, :, :L] = x.transpose(0, 1)
    y.masked_fill_((torch.arange(N * CHUNK, device=x.device) >= lens[:, None])[None, :, :, None], 0.0)
    return y.view(H, B, N, CHUNK, d)


class _Plain:
    """The chunkwise form's decays: [H, B, N, ..] with n[b, c] tokens in chunk c of sequence b."""

    def __init__(self, s):
        B, H, L, d = s["q"].shape
        dev = s["q"].device
        self.shape, self.type, self.scale = (B, H, L, d), s["q"].dtype, 1.0 / math.sqrt(d)
        self.lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), L, device=dev)
        N = -(-L // CHUNK)
        i = torch.arange(CHUNK, device=dev)
        self.n = (self.lens[:, None] - CHUNK * torch.arange(N, device=dev)).clamp(0, CHUNK)  # [B, N]
        g = s["g"][:, None, None, None]
        m = i[:, None] - i[None, :]
        self.inner = torch.where(m >= 0, _power(g, m.clamp(min=0)[None, None]), 0.0)[:, :, None]  # [H, 1, 1, C, C]
        self.from_start = _power(g, (i + 1)[None, None])[..., None]
        to_end = self.n[..., None] - 1 - i
        self.to_end = torch.where(to_end >= 0, _power(g, to_end.clamp(min=0)), 0.0)[..., None]
        self.whole = _power(g, self.n[..., None])  # [H, B, N, 1]

    def back(self, y):
        """[H, B, N, C, d] as [B, H, L, d] in the inputs' type, zero behind a sequence's end."""
        B, H, L, d = self.shape
        return self._cut(y.reshape(H, B, -1, d)).transpose(0, 1).contiguous().to(self.type)

    def _cut(self, y):
        L = self.shape[2]
        return y[:, :, :L].masked_fill((torch.arange(L, device=y.device) >= self.lens[:, None])[None, :, :, None], 0.0)

    def states(self, k, v, state):
        """State [dv, dk] ahead of each chunk, and the last one."""
        B, H, _, d = self.shape
        add = (v * self.to_end).transpose(-1, -2) @ k
        at = torch.zeros((H, B, d, d), device=k.device) if state is None else state.transpose(0, 1)
        before = []
        for c in range(add.shape[2]):
            before.append(at)
            at = self.whole[:, :, c, :, None] * at + add[:, :, c]
        return torch.stack(before, 2), at

    def states_back(self, q, u, dstate):
        """The same from the other end: the state's gradient behind each chunk, and that of the first state."""
        B, H, _, d = self.shape
        add = (u * (self.from_start * self.scale)).transpose(-1, -2) @ q
        at = torch.zeros((H, B, d, d), device=q.device) if dstate is None else dstate.transpose(0, 1)
        behind = [None] * add.shape[2]
        for c in reversed(range(add.shape[2])):
            behind[c] = at
            at = self.whole[:, :, c, :, None] * at + add[:, :, c]
        return torch.stack(behind, 2), at


def _plain_attn(s):
    p = _Plain(s)
    q, k, v = (_chunks(s[n], p.lens) for n in "qkv")
    before, last = p.states(k, v, s["state"])
    o = ((q @ k.transpose(-1, -2)) * p.inner) @ v
    o = (o + (q @ before.transpose(-1, -2)) * p.from_start) * p.scale
    out = p.back(o)
    return (out, last.transpose(0, 1).contiguous()) if s["case"]["state"] else out


def _plain_attn_grad(s):
    p = _Plain(s)
    q, k, v, u = (_chunks(s[n], p.lens) for n in ("q", "k", "v", "dout"))
    before, _ = p.states(k, v, s["state"])
    behind, first = p.states_back(q, u, s["dstate"])
    dp = (u @ v.transpose(-1, -2)) * (p.inner * p.scale)
    dq = dp @ k + (u @ before) * (p.from_start * p.scale)
    dk = dp.transpose(-1, -2) @ q + (v @ behind) * p.to_end
    dp = (q @ k.transpose(-1, -2)) * (p.inner * p.scale)
    dv = dp.transpose(-1, -2) @ u + (k @ behind.transpose(-1, -2)) * p.to_end
    out = tuple(p.back(y) for y in (dq, dk, dv))
    return out + (first.transpose(0, 1).contiguous(),) if s["case"]["state"] else out


def _plain_step(s):
    q, k, v = (s[n].to(torch.float32) for n in "qkv")
    S = s["state"]
    S.mul_(torch.exp(s["g"])[None, :, None, None]).add_(v[..., :, None] * k[..., None, :])
    o = (S @ q[..., None])[..., 0] / math.sqrt(q.shape[-1])
    return o.to(s["q"].dtype), S


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s["x"], s["w"], s["b"])
    if op == "norm_grad":
        return _plain_norm_grad(s["dy"], s["x"], s["w"])
    return {"attn": _plain_attn, "attn_grad": _plain_attn_grad, "step": _plain_step}[op](s)


# ------------------------------------------------------------ the operators

def _own(s):
    import linear_attention_nats_gb300 as nats

    c = s["case"]
    if c["op"] == "norm":
        return nats.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
    if c["op"] == "norm_grad":
        r = nats.layer_norm_bwd(s["dy"], s["x"], s["w"], eps=EPS)
        return r["dx"], r["dw"], r["db"]
    if c["op"] == "attn":
        return nats.decay_attn(s["q"], s["k"], s["v"], s["g"], lens=s["lens"], state=s["state"], return_state=c["state"])
    if c["op"] == "attn_grad":
        r = nats.decay_attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["g"], lens=s["lens"], state=s["state"],
                                dstate_out=s["dstate"], state_grad=c["state"])
        return (r["dq"], r["dk"], r["dv"]) + ((r["dstate"],) if c["state"] else ())
    return nats.decay_attn_step(s["q"], s["k"], s["v"], s["g"], s["state"]), s["state"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- values in 64 bits

def _exact_norm(x, w, b):
    D = x.shape[-1]
    x = x.double()
    mu = x.sum(-1, keepdim=True) / D
    var = ((x - mu) ** 2).sum(-1, keepdim=True) / D
    return (x - mu) * (var + EPS) ** -0.5 * w.double() + b.double()


def _exact_norm_grad(dy, x, w):
    """The vector-Jacobian product of y = w xc / n, xc = x - mean(x), n = sqrt(|xc|^2 / D + eps):
    with t = w dy / n, the part of t along xc taken out, dx = (t - xc <t, xc> / (D n^2)) less its mean."""
    D = x.shape[-1]
    xc = x.double() - x.double().sum(-1, keepdim=True) / D
    n2 = (xc * xc).sum(-1, keepdim=True) / D + EPS
    u = dy.double()
    t = u * w.double() * n2 ** -0.5
    t = t - xc * ((t * xc).sum(-1, keepdim=True) / (D * n2))
    dx = t - t.sum(-1, keepdim=True) / D
    u, z = u.reshape(-1, D), (xc * n2 ** -0.5).reshape(-1, D)
    return dx, torch.einsum("nd,nd->d", u, z), u.sum(0)


def _exact_attn(s):
    """S_t = e^g S_(t-1) + v_t k_t^T, o_t = S_t q_t / sqrt(d), token by token."""
    q, k, v = (s[n].double() for n in "qkv")
    B, H, L, d = q.shape
    a = torch.exp(s["g"].double())[None, :, None, None]
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].double()
    out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    lens = s["lens"].long() if s["lens"] is not None else None
    for t in range(L):
        S1 = torch.addcmul(S * a, v[:, :, t, :, None], k[:, :, t, None, :])
        o = (S1 * q[:, :, t, None, :]).sum(-1) if d * B * H < 65536 else torch.matmul(S1, q[:, :, t, :, None])[..., 0]
        if lens is None:
            S, out[:, :, t] = S1, o
        else:
            live = (t < lens)[:, None, None]
            S = torch.where(live[..., None], S1, S)
            out[:, :, t] = torch.where(live, o, 0.0)
    out /= math.sqrt(d)
    return (out, S) if s["case"]["state"] else out


def _exact_attn_grad(s):
    """R_t, the gradient of S_t: R_t = u_t q_t^T / sqrt(d) + e^g R_(t+1), from dstate down; dq_t = S_t^T u_t / sqrt(d),
    dk_t = R_t^T v_t, dv_t = R_t k_t, and e^g R_1 for the first state."""
    q, k, v, u = (s[n].double() for n in ("q", "k", "v", "dout"))
    B, H, L, d = q.shape
    a = torch.exp(s["g"].double())[None, :, None, None]
    lens = s["lens"].tolist() if s["lens"] is not None else [L] * B
    live = [torch.tensor([float(t < n) for n in lens], dtype=torch.float64, device=DEV)[:, None, None, None] for t in
            range(L)] if s["lens"] is not None else None
    u = u / math.sqrt(d)
    S = torch.zeros(B, H, d, d, dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].double()
    dq, dk, dv = (torch.zeros_like(q, memory_format=torch.contiguous_format) for _ in range(3))
    for t in range(L):
        # (a sequence that has ended is not asked for its state again)
        S = torch.addcmul(S * a, v[:, :, t, :, None], k[:, :, t, None, :])
        dq[:, :, t] = torch.matmul(u[:, :, t, None, :], S)[:, :, 0]
    R = torch.zeros_like(S) if s["dstate"] is None else s["dstate"].double()
    for t in reversed(range(L)):
        R1 = torch.addcmul(R, u[:, :, t, :, None], q[:, :, t, None, :])
        dk[:, :, t] = torch.matmul(v[:, :, t, None, :], R1)[:, :, 0]
        dv[:, :, t] = torch.matmul(R1, k[:, :, t, :, None])[..., 0]
        R = R1 * a if live is None else torch.where(live[t] > 0, R1 * a, R)
    if live is not None:
        alive = torch.stack(live)[:, :, :, 0].permute(1, 2, 0, 3)
        dq, dk, dv = (torch.where(alive > 0, y, 0.0) for y in (dq, dk, dv))
    return (dq, dk, dv, R) if s["case"]["state"] else (dq, dk, dv)


def _exact_step(s):
    q, k, v = (s[n].double() for n in "qkv")
    S = s["state"].double() * torch.exp(s["g"].double())[None, :, None, None]
    S = S + torch.einsum("bhi,bhj->bhij", v, k)
    return torch.einsum("bhij,bhj->bhi", S, q) / math.sqrt(q.shape[-1]), S


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s["x"], s["w"], s["b"])
    if case["op"] == "norm_grad":
        return _exact_norm_grad(s["dy"], s["x"], s["w"])
    if case["op"] == "step":
        return _exact_step(s)
    # (token by token: about 8 s for 131,072 tokens of 8 heads)
    if case["B"] * case["H"] * case["L"] * case["d"] ** 2 > 2 ** 35 or case["L"] > 140000:
        return None
    return _exact_attn(s) if case["op"] == "attn" else _exact_attn_grad(s)
