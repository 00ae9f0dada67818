"""The README's decode step, line by line as it stands there."""

import os
import re

import pytest
import torch

import serving_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_decode_step():
    from linear_attention_nats_gb300 import build

    build.build()
    import linear_attention_nats_gb300 as nats

    text = open(os.path.join(ROOT, "README.md")).read()
    lines = re.search(r"A decode step of a softmax layer over the paged cache:\n\n((?:    .*\n)+)", text).group(1)
    lines = [x[4:] for x in lines.splitlines()]
    step = lines.index(next(x for x in lines if "paged_append" in x))
    behind = lines.index(next(x for x in lines if x.startswith("#")))
    B, Hq, Hk, max_pages, steps = 2, 8, 2, 40, 3
    n_pages = 2 * B * max_pages
    rng = torch.Generator().manual_seed(1)
    order = torch.randperm(n_pages, generator=rng).to(torch.int32).cuda()
    env = dict(nats=nats, n_pages=n_pages, Hk=Hk, B=B, max_pages=max_pages, table=order[:B * max_pages].view(B, max_pages),
               fresh_table=order[B * max_pages:].view(B, max_pages).contiguous(), w_q=None, w_k=None)
    exec("\n".join(lines[:step]), env)
    c = env["cache"]
    for t in range(steps):
        q, k, v = (torch.randn(B, h, 1, 128, generator=rng).to(torch.bfloat16).cuda() for h in (Hq, Hk, Hk))
        env.update(q=q, k=k, v=v, pos=torch.full((B, 1), t, device="cuda"))
        exec("\n".join(lines[step:behind]), env)
        assert c.lens.tolist() == [t + 1] * B
        e, _, _, err, _ = ref.decode(env["q"][:, :, 0].cpu(), c.k_pages.cpu(), c.v_pages.cpu(), c.table.cpu(), c.lens.tolist())
        assert ((env["out"].cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()
    # a sequence longer than the budget, its slots as they came
    c.lens.copy_(torch.tensor([2500, 2048], dtype=torch.int32))
    c.weight.copy_(torch.rand(c.weight.shape, generator=rng))
    want = ref.evict(c.weight.cpu(), c.table.cpu(), [2500, 2048], 64, 2048, 256, 4)
    was, old = c.k_pages.cpu(), c.table.cpu()
    exec("\n".join(lines[behind:]), env)
    c.check()
    assert c.lens.tolist() == [2048, 2048] and torch.equal(c.table, env["fresh_table"])
    got = c.k_pages.cpu()
    for b in range(B):
        for h in range(Hk):
            src = want[b, h].long()
            assert torch.equal(ref.slots(got, c.table.cpu(), b, 2048, 64)[h], was[old[b].long()[src // 64], h, src % 64])
