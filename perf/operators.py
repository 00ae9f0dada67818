"""Cases, plain forms and 64-bit values of the serving operators around the
attention layers: the norm and rotation of queries and keys (and its
gradient), the paged key / value cache's append, the attention of one new
token over it, and its eviction by accumulated attention weight.

`own` chooses what `run` computes with: elementary torch operations in fp32,
or the library's operators.
"""

import math

import torch

own = False

DEV = "cuda"
BASE = 1.0e6  # rotation base of long-context models
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of one sequence, far into its context: launch latency
        dict(name="rope token", op="rope", B=1, L=1, Hq=16, Hk=16, d=128, rot=128, pairs="half", type="bf16", start=131072),
        # the layer's 1.3B-scale prefill (B 4, H 16, L 8192), q and k inside one projection's output
        dict(name="rope prefill", op="rope", B=4, L=8192, Hq=16, Hk=16, d=128, rot=128, pairs="half", type="bf16", start=0),
        # its training step: fp32 gradients as the layer's backward gives them, into one bf16 gradient buffer
        dict(name="rope gradient", op="rope_grad", B=4, L=8192, Hq=16, Hk=16, d=128, rot=128, pairs="half", type="bf16",
             grad="f32", start=0),
        # an odd fp32 shape: shared key heads, a partial rotation of neighbouring pairs
        dict(name="rope gradient f32", op="rope_grad", B=3, L=1021, Hq=12, Hk=4, d=64, rot=32, pairs="next", type="f32",
             grad="f32", start=77),
        # a decode batch's new tokens: norm, rotation and append in one call
        dict(name="append tokens", op="append", B=32, T=1, Hq=32, Hk=8, d=128, rot=128, pairs="half", type="bf16", page=64,
             start=8191, norm=True),
        # a ragged batch of prompts into the cache
        dict(name="append prompts", op="append", B=8, T=4096, Hq=32, Hk=8, d=128, rot=128, pairs="half", type="bf16",
             page=64, start=0, norm=True),
        # one short conversation, one key head for each query head
        dict(name="decode short", op="decode", B=1, len=517, Hq=16, Hk=16, d=128, type="bf16", page=64, weights=False),
        # a serving batch of ragged contexts up to 8192 tokens, four query heads to a key head
        dict(name="decode batch", op="decode", B=32, len=8192, Hq=32, Hk=8, d=128, type="bf16", page=64, weights=False),
        # the 131,072-token context, with the weights that eviction goes by
        dict(name="decode long", op="decode", B=4, len=131072, Hq=32, Hk=8, d=128, type="bf16", page=64, weights=True),
        # fp32, small pages, an odd batch with empty and one-token sequences
        dict(name="decode f32", op="decode", B=17, len=3001, Hq=12, Hk=4, d=64, type="f32", page=16, weights=True),
        # a cache held at 2048 tokens, shortened every 64 steps
        dict(name="evict step", op="evict", B=32, len=2112, Hk=8, d=128, type="bf16", page=64, budget=2048, recent=256, sinks=4),
        # a long prompt's cache brought down to a quarter
        dict(name="evict long", op="evict", B=4, len=131072, Hk=8, d=128, type="bf16", page=64, budget=32768, recent=1024,
             sinks=4),
    ]


MOST_BYTES = 1 << 30  # of a drawn case's pass; the largest listed one has about 2^31


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "rope_grad", "append", "decode", "decode", "evict"])
        t = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 3, 4, 6, 8, 16])
        G = rng.choice([1, 1, 2, 3, 4, 5, 8, 12])
        rope = dict(d=d, rot=rng.choice([d, d, d // 2, d - 16]), pairs=rng.choice(["half", "half", "next"]))
        if op in ("rope", "rope_grad"):
            c = dict(op=op, B=_log(rng, 1, 16), L=_log(rng, 1, 16384), Hq=Hk * G, Hk=Hk, type=t, start=_log(rng, 1, 1000000), **rope)
            if op == "rope_grad":
                c["grad"] = "f32" if t == "f32" else rng.choice(["f32", "bf16"])
        elif op == "append":
            c = dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 8192), Hq=Hk * G, Hk=Hk, type=t, page=rng.choice([16, 32, 48, 64, 128]),
                     start=_log(rng, 1, 8192), norm=rng.random() < 0.75, **rope)
        elif op == "decode":
            c = dict(op=op, B=_log(rng, 1, 256), len=_log(rng, 1, 262144), Hq=Hk * G, Hk=Hk, d=d, type=t,
                     page=rng.choice([16, 32, 48, 64, 128]), weights=rng.random() < 0.5)
        else:
            n = _log(rng, 64, 131072)
            c = dict(op=op, B=_log(rng, 1, 64), len=n, Hk=Hk, d=d, type=t, page=rng.choice([16, 32, 48, 64, 128]),
                     budget=rng.randint(n // 4, n), recent=0, sinks=rng.choice([0, 1, 4]))
            c["budget"] = max(8, c["budget"])
            c["recent"] = rng.randint(0, (c["budget"] - c["sinks"]) // 2)
        if work(c)["bytes"] <= MOST_BYTES and _held(c) <= 4 * MOST_BYTES:
            return c


def _es(c):
    return 2 if c["type"] == "bf16" else 4


def _lens(c):
    """The batch's lengths: the case's own first, then shorter ones, an empty and a one-token sequence among them."""
    n, B = c["len"] if "len" in c else c["T"], c["B"]
    lens = [n - (n * 7 * b // (11 * B)) for b in range(B)]
    if B >= 16 and c.get("op") != "evict":
        lens[B // 2], lens[B // 3] = 0, 1
    return lens


def _held(c):
    """Bytes of the cache pages (or of the projection's output) that the case's state holds."""
    if "page" in c:
        n = c["len"] if "len" in c else c["start"] + c["T"]
        return c["B"] * (n + c["page"]) * c["Hk"] * c["d"] * _es(c) * 2 * (2 if c["op"] == "evict" else 1)
    return c["B"] * c["L"] * (c["Hq"] + 2 * c["Hk"]) * c["d"] * _es(c) * 2


def work(c):
    es, d = _es(c), c["d"]
    if c["op"] == "rope":
        n = c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * d
        return dict(bytes=2 * n * es + c["B"] * c["L"] * 8, flops=8 * n)
    if c["op"] == "rope_grad":
        n = c["B"] * c["L"] * (c["Hq"] + c["Hk"]) * d
        return dict(bytes=n * (2 * es + (4 if c["grad"] == "f32" else 2)) + c["B"] * c["L"] * 8 + 16 * d, flops=18 * n)
    if c["op"] == "append":
        rows = sum(_lens(c))
        n = rows * (c["Hq"] + 2 * c["Hk"]) * d
        return dict(bytes=2 * n * es + rows * (8 + 4 * c["Hk"]), flops=8 * rows * (c["Hq"] + c["Hk"]) * d)
    if c["op"] == "decode":
        rows = sum(_lens(c))
        n = rows * c["Hk"]
        return dict(bytes=2 * n * d * es + 2 * c["B"] * c["Hq"] * d * es + (8 * n if c["weights"] else 0),
                    flops=4 * rows * c["Hq"] * d)
    rows = sum(_lens(c))
    kept = sum(min(n, c["budget"]) for n in _lens(c))
    return dict(bytes=c["Hk"] * (4 * rows + kept * (4 * d * es + 8)), flops=c["Hk"] * rows)


# ------------------------------------------------------------------ inputs

def _cache(c, lens, gen, pool_extra=0, spread=1.0):
    """Pages in a shuffled order, a page table (-1 behind a sequence's pages) and the lengths."""
    B, page, dt = c["B"], c["page"], TYPES[c["type"]]
    cap = [max(1, -(-n // page)) for n in lens]
    n_pages = sum(cap) + pool_extra
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((B, max(cap)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(cap):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (n_pages, c["Hk"], page, c["d"])
    k = torch.randn(shape, generator=gen, device=DEV, dtype=dt)
    v = torch.randn(shape, generator=gen, device=DEV, dtype=dt)
    lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return dict(k=k, v=v, table=table, lens=lens_t, spare=order[at:], n=max(lens))


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=c)
    d = c["d"]
    dt = TYPES[c["type"]]
    randn = lambda *shape, dtype=torch.float32: torch.randn(shape, generator=gen, device=DEV, dtype=dtype)
    if c["op"] in ("rope", "rope_grad", "append"):
        B, T, Hq, Hk = c["B"], c["L"] if "L" in c else c["T"], c["Hq"], c["Hk"]
        W = (Hq + 2 * Hk) * d
        s["qkv"] = randn(B, T, W, dtype=dt)
        s["q"], s["k"], s["v"] = _heads(s["qkv"], Hq, Hk, d)
        s["w_q"], s["w_k"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
        r = c["rot"]
        s["inv_freq"] = torch.tensor([BASE ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device=DEV)
        if c["op"] != "append":
            first = c["start"] + torch.arange(B, device=DEV) * 13
            s["pos"] = first[:, None] + torch.arange(T, device=DEV)[None]
        if c["op"] == "rope_grad":
            gt = TYPES[c["grad"]]
            s["dq_out"], s["dk_out"] = randn(B, Hq, T, d, dtype=gt), randn(B, Hk, T, d, dtype=gt)
            s["dqkv"] = torch.zeros_like(s["qkv"])
            s["dq"], s["dk"], _ = _heads(s["dqkv"], Hq, Hk, d)
    if c["op"] == "append":
        n_new = _lens(c)
        start = [max(0, c["start"] - 5 * b) for b in range(B)]
        m = _cache(c, [p + T for p in start], gen)
        s["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        s["n_new"] = torch.tensor(n_new, dtype=torch.int32, device=DEV)
        s["out_q"] = torch.zeros((B, Hq, T, d), dtype=dt, device=DEV)
        s["weight"] = randn(m["k"].shape[0], Hk, c["page"]).abs()
    elif c["op"] == "decode":
        m = _cache(c, _lens(c), gen)
        s["q"] = 2 * randn(c["B"], c["Hq"], d)
        s["q"] = s["q"].to(dt)
        s["weight"] = randn(m["k"].shape[0], c["Hk"], c["page"]).abs() if c["weights"] else None
    elif c["op"] == "evict":
        lens = _lens(c)
        per = -(-c["budget"] // c["page"])
        m = _cache(c, lens, gen, pool_extra=per * c["B"])
        s["out_table"] = m["spare"].reshape(c["B"], per).contiguous()
        # attention gathers on few tokens; the newest have had none yet
        w = torch.exp(2 * randn(m["k"].shape[0], c["Hk"], c["page"]))
        s["weight"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.1, torch.zeros_like(w), w)
    if "page" in c:
        s["m"] = m
        if own:  # the handle that a serving program keeps for its cache
            import linear_attention_nats_gb300 as nats

            s["cache"] = nats.PagedCache(m["k"], m["v"], m["table"], m["lens"], weight=s["weight"])
            if c["op"] != "append":
                s["ws"] = torch.empty(nats.paged_workspace_size(s["cache"], Hq=c.get("Hq", 0), accumulate=c.get("weights", False),
                                                                budget=c.get("budget", 0)), dtype=torch.uint8, device=DEV)
    return s


def _heads(qkv, Hq, Hk, d):
    """q, k, v [B, H, T, d] inside a projection's output [B, T, (Hq + 2 Hk) d]."""
    B, T, _ = qkv.shape
    q = qkv[..., :Hq * d].view(B, T, Hq, d).transpose(1, 2)
    k = qkv[..., Hq * d:(Hq + Hk) * d].view(B, T, Hk, d).transpose(1, 2)
    v = qkv[..., (Hq + Hk) * d:].view(B, T, Hk, d).transpose(1, 2)
    return q, k, v


# ------------------------------------------------------------- plain forms

def _angles(pos, inv_freq):
    """cos and sin [B, 1, T, r / 2]; the angle in 64 bits, for far positions."""
    a = pos.double()[:, None, :, None] * inv_freq
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, pairs):
    r = 2 * cos.shape[-1]
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _norm_rotate(x, w, cos, sin, pairs):
    x = x.float()
    return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w, cos, sin, pairs)


def _norm_rotate_grad(dy, x, w, cos, sin, pairs):
    x = x.float()
    u = _rotate(dy.float(), cos, -sin, pairs)
    rs = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * rs
    g = u * w
    dx = rs * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (u * xh).sum((0, 1, 2))


def _rows(pages, table, n):
    """Rows 0 .. n - 1 of every sequence and head, in order: [B, H, n, ...]."""
    npg = -(-n // pages.shape[2])
    x = pages[table[:, :npg].long().clamp(min=0)].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], npg * pages.shape[2], *pages.shape[3:])[:, :, :n]


def _put(pages, page, slot, rows, valid):
    """rows [B, H, n, ...] to pages[page[b, n], h, slot[b, n]] where valid [B, 1, n]."""
    h = torch.arange(pages.shape[1], device=pages.device)[None, :, None]
    at = (page[:, None, :], h, slot[:, None, :])
    valid = valid if rows.dim() == 3 else valid[..., None]
    pages[at] = torch.where(valid, rows.to(pages.dtype), pages[at])


def _plain_append(s):
    c, m = s["case"], s["m"]
    T = c["T"]
    t = torch.arange(T, device=DEV)
    at = s["start"].long()[:, None] + t
    valid = (t < s["n_new"][:, None])[:, None, :]
    q, k = s["q"], s["k"]
    if c["norm"]:
        cos, sin = _angles(at, s["inv_freq"])
        q, k = _norm_rotate(q, s["w_q"], cos, sin, c["pairs"]), _norm_rotate(k, s["w_k"], cos, sin, c["pairs"])
    page, slot = m["table"].gather(1, at // c["page"]).long(), at % c["page"]
    _put(m["k"], page, slot, k, valid)
    _put(m["v"], page, slot, s["v"], valid)
    _put(s["weight"], page, slot, torch.zeros(k.shape[:3], device=DEV), valid)
    s["out_q"].copy_(torch.where(valid[..., None], q.to(s["out_q"].dtype), s["out_q"]))
    return s["out_q"], m["k"], m["v"], s["weight"]


def _plain_decode(s):
    c, m = s["case"], s["m"]
    B, Hq, d = s["q"].shape
    Hk, n = c["Hk"], max(1, m["n"])
    k, v = _rows(m["k"], m["table"], n).float(), _rows(m["v"], m["table"], n).float()
    q = s["q"].float().view(B, Hk, Hq // Hk, d) * d ** -0.5
    x = q @ k.transpose(2, 3)
    seen = torch.arange(n, device=DEV) < m["lens"][:, None, None, None]
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.where(seen, torch.exp(x - top), 0.0)
    total = e.sum(-1, keepdim=True)
    p = e / total.clamp(min=1e-37)
    out = (p @ v).to(s["q"].dtype).view(B, Hq, d)
    if not c["weights"]:
        return out
    at = torch.arange(n, device=DEV)[None].expand(B, n)
    page, slot = m["table"].gather(1, at // c["page"]).long().clamp(min=0), at % c["page"]
    h = torch.arange(Hk, device=DEV)[None, :, None]
    # rows behind a sequence add nothing, wherever their table entry points
    flat = (page[:, None, :] * Hk + h) * c["page"] + slot[:, None, :]
    s["weight"].view(-1).scatter_add_(0, flat.reshape(-1), p.sum(2).reshape(-1))
    return out, s["weight"]


def _plain_evict(s):
    c, m = s["case"], s["m"]
    n, K = m["n"], c["budget"]
    w = _rows(s["weight"], m["table"], n)
    B, Hk, _ = w.shape
    lens = m["lens"].long()[:, None, None]
    j = torch.arange(n, device=DEV)
    always = (j < c["sinks"]) | (j >= lens - c["recent"])
    key = torch.where(always, float("inf"), w)
    key = torch.where(j < lens, key, float("-inf"))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    left = lens.clamp(max=K)
    i = torch.arange(min(n, K), device=DEV)
    valid = i < left  # [B, 1, K']
    keep = torch.where(valid, order[..., :min(n, K)], n).sort(dim=-1).values
    src = keep.clamp(max=n - 1)
    out_page, out_slot = s["out_table"].long()[:, i // c["page"]], (i % c["page"]).expand(B, -1)
    page, slot = m["table"].long()[:, None, :].expand(B, Hk, -1).gather(2, src // c["page"]), src % c["page"]
    h = torch.arange(Hk, device=DEV)[None, :, None]
    for pages in (m["k"], m["v"], s["weight"]):
        _put(pages, out_page, out_slot, pages[page, h, slot], valid)
    keep = torch.where(valid, keep, -1).to(torch.int32)
    if K > n:
        keep = torch.cat([keep, torch.full((B, Hk, K - n), -1, dtype=torch.int32, device=DEV)], -1)
    return keep, left[:, 0, 0].to(torch.int32), m["k"], m["v"], s["weight"]


def _plain(s):
    c = s["case"]
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "decode":
        return _plain_decode(s)
    if c["op"] == "evict":
        return _plain_evict(s)
    cos, sin = _angles(s["pos"], s["inv_freq"])
    if c["op"] == "rope":
        dt = s["q"].dtype
        return (_norm_rotate(s["q"], s["w_q"], cos, sin, c["pairs"]).to(dt),
                _norm_rotate(s["k"], s["w_k"], cos, sin, c["pairs"]).to(dt))
    dq, dw_q = _norm_rotate_grad(s["dq_out"], s["q"], s["w_q"], cos, sin, c["pairs"])
    dk, dw_k = _norm_rotate_grad(s["dk_out"], s["k"], s["w_k"], cos, sin, c["pairs"])
    s["dq"].copy_(dq)
    s["dk"].copy_(dk)
    return s["dq"], s["dk"], dw_q, dw_k


# ------------------------------------------------------------ the operators

def _own(s):
    import linear_attention_nats_gb300 as nats

    c = s["case"]
    if c["op"] == "rope":
        return nats.qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"], interleaved=c["pairs"] == "next",
                                 eps=EPS)
    if c["op"] == "rope_grad":
        g = nats.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["pos"],
                                  interleaved=c["pairs"] == "next", eps=EPS, dq=s["dq"], dk=s["dk"])
        return g["dq"], g["dk"], g["dw_q"], g["dw_k"]
    if c["op"] == "append":
        if c["norm"]:
            nats.paged_append(s["cache"], s["k"], s["v"], start=s["start"], n_new=s["n_new"], q=s["q"], out_q=s["out_q"],
                              norm=True, w_q=s["w_q"], w_k=s["w_k"], inv_freq=s["inv_freq"],
                              interleaved=c["pairs"] == "next", eps=EPS)
        else:
            nats.paged_append(s["cache"], s["k"], s["v"], start=s["start"], n_new=s["n_new"], q=s["q"], out_q=s["out_q"])
        return s["out_q"], s["m"]["k"], s["m"]["v"], s["weight"]
    if c["op"] == "decode":
        out = nats.paged_decode(s["cache"], s["q"], accumulate=c["weights"], workspace=s["ws"])
        return (out, s["weight"]) if c["weights"] else out
    keep, lens = nats.paged_evict(s["cache"], s["out_table"], c["budget"], recent=c["recent"], sinks=c["sinks"],
                                  return_keep=True, workspace=s["ws"])
    return keep, lens, s["m"]["k"], s["m"]["v"], s["weight"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- values in 64 bits

def _unit(c, pos, s):
    """The rotation as complex factors [B, 1, T, r / 2]."""
    a = pos.to(torch.float64)[:, None, :, None] * s["inv_freq"]
    return torch.polar(torch.ones_like(a), a)


def _turn(x, z, pairs):
    """x [..., d] in 64 bits with its first r entries, taken as complex numbers, times z."""
    r = 2 * z.shape[-1]
    head = x[..., :r].reshape(*x.shape[:-1], 2, r // 2).movedim(-2, -1) if pairs == "half" else x[..., :r].reshape(*x.shape[:-1], r // 2, 2)
    t = torch.view_as_real(torch.view_as_complex(head.contiguous()) * z)
    t = t.movedim(-1, -2) if pairs == "half" else t
    return torch.cat([t.reshape(*x.shape[:-1], r), x[..., r:]], -1)


def _exact_rows(x, w, z, pairs):
    x = x.to(torch.float64)
    return _turn(x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double(), z, pairs)


def _exact_grad(dy, x, w, z, pairs):
    """From d/dx of y = R (w x / n), n = sqrt(|x|^2 / d + eps): dx = (w u - x <w u, x> / (d n^2)) / n, u = R^T dy."""
    x, u = x.to(torch.float64), _turn(dy.to(torch.float64), z.conj(), pairs)
    n = torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    dw = torch.einsum("bhtd,bhtd->d", u, x / n)
    u = u * w.double()
    return (u - x * ((u * x).sum(-1, keepdim=True) / (x.shape[-1] * n * n))) / n, dw


def exact(case, seed):
    s = prepare(case, seed)
    c, m = s["case"], s.get("m")
    if c["op"] == "rope":
        z = _unit(c, s["pos"], s)
        return tuple(_exact_rows(s[n], s["w_" + n], z, c["pairs"]) for n in ("q", "k"))
    if c["op"] == "rope_grad":
        z = _unit(c, s["pos"], s)
        (dq, dwq), (dk, dwk) = (_exact_grad(s["d%s_out" % n], s[n], s["w_" + n], z, c["pairs"]) for n in ("q", "k"))
        return dq, dk, dwq, dwk
    page = c["page"]
    if c["op"] == "append":
        out_q, kp, vp, w = s["out_q"].double(), m["k"].double(), m["v"].double(), s["weight"].double()
        start, n_new = s["start"].tolist(), s["n_new"].tolist()
        for b in range(c["B"]):
            n = n_new[b]
            if n == 0:
                continue
            pos = torch.arange(start[b], start[b] + n, device=DEV)
            q, k = s["q"][b:b + 1, :, :n].double(), s["k"][b:b + 1, :, :n].double()
            if c["norm"]:
                z = _unit(c, pos[None], s)
                q, k = _exact_rows(q, s["w_q"], z, c["pairs"]), _exact_rows(k, s["w_k"], z, c["pairs"])
            pg, sl = m["table"][b].long()[pos // page], pos % page
            out_q[b, :, :n] = q[0]
            kp[pg, :, sl] = k[0].transpose(0, 1)
            vp[pg, :, sl] = s["v"][b, :, :n].double().transpose(0, 1)
            w[pg, :, sl] = 0
        return out_q, kp, vp, w
    lens = m["lens"].tolist()
    if c["op"] == "decode":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        w = s["weight"].double() if c["weights"] else None
        G = c["Hq"] // c["Hk"]
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pg = m["table"][b, :-(-n // page)].long()
            k = m["k"][pg].double().transpose(0, 1).reshape(c["Hk"], -1, c["d"])[:, :n]
            v = m["v"][pg].double().transpose(0, 1).reshape(c["Hk"], -1, c["d"])[:, :n]
            q = s["q"][b].double().view(c["Hk"], G, c["d"])
            p = torch.softmax(torch.bmm(q, k.transpose(1, 2)) / math.sqrt(c["d"]), -1)
            out[b] = torch.bmm(p, v).reshape(c["Hq"], c["d"])
            if c["weights"]:
                j = torch.arange(n, device=DEV)
                w[pg[j // page], :, j % page] += p.sum(1).transpose(0, 1)
        return (out, w) if c["weights"] else out
    # eviction moves rows: its values are the inputs' own
    K = c["budget"]
    keep = torch.full((c["B"], c["Hk"], K), -1, dtype=torch.int32, device=DEV)
    kp, vp, w = m["k"].clone(), m["v"].clone(), s["weight"].clone()
    for b, n in enumerate(lens):
        left = min(n, K)
        pg = m["table"][b, :-(-n // page)].long()
        wt = s["weight"][pg].transpose(0, 1).reshape(c["Hk"], -1)[:, :n].double()
        kept = torch.zeros((c["Hk"], n), dtype=torch.bool, device=DEV)
        if n <= K:
            kept[:] = True
        else:
            kept[:, :c["sinks"]] = True
            kept[:, n - c["recent"]:] = True
            free = K - c["sinks"] - c["recent"]
            mid = wt[:, c["sinks"]:n - c["recent"]]
            best = mid.neg().argsort(dim=-1, stable=True)[:, :free]
            kept[:, c["sinks"]:n - c["recent"]] |= torch.zeros_like(mid, dtype=torch.bool).scatter(1, best, True)
        idx = kept.nonzero()[:, 1].view(c["Hk"], left)
        keep[b, :, :left] = idx
        i = torch.arange(left, device=DEV)
        h = torch.arange(c["Hk"], device=DEV)[:, None]
        to = (s["out_table"][b].long()[i // page][None], h, (i % page)[None])
        fr = (pg[idx // page], h, idx % page)
        kp[to], vp[to], w[to] = m["k"][fr], m["v"][fr], s["weight"][fr]
    return keep, torch.tensor([min(n, K) for n in lens], dtype=torch.int32, device=DEV), kp, vp, w
