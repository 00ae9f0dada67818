"""The paged cache next to the framework's own layer."""

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


@pytest.mark.parametrize("H,d,sel", [(2, 64, [0, 0, 0, 0, 0]), (4, 128, [0, 1, 0, 1, 0])])
def test_decode_over_a_layers_prompt_is_its_softmax_branch(nats, H, d, sel):
    """A prompt through norm + rotation into the hybrid layer and, by paged_append, into a cache of one chunk a page.
    A token of the layer's softmax branch attends to the softmax-selected chunks before its own, and causally to its
    own: paged_decode over the pages of those chunks gives the same row and log-sum-exp (the layer's bar: 1e-2 of the
    largest entry; its log2 of the sum of weights each off by 1e-2 at most)."""
    L = 64 * len(sel)
    rng = torch.Generator().manual_seed(d)
    qkv = torch.randn(1, L, 3, H, d, generator=rng).to(BF).cuda()
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    f = nats.rope_inv_freq(d)
    wk = torch.full((d,), d ** -0.5, device="cuda")  # unit keys
    q2, k2 = nats.qk_norm_rope(q, k, None, wk, f)
    g, beta = -0.1 * torch.rand(1, H, L, generator=rng), torch.rand(1, H, L, generator=rng)
    codes = torch.tensor(sel, dtype=torch.uint8).expand(1, H, -1).contiguous().cuda()
    layer = nats.hybrid_fwd(q2, k2, v.contiguous(), g.cuda(), beta.cuda(), None, None,
                            0.02 * torch.randn(H, d, generator=rng).cuda(), sel_in=codes, scale=1.0, return_branches=True,
                            return_lse=True)
    pool = nats.PagedCache.empty(len(sel), 64, H, d, 1, len(sel))
    order = torch.randperm(len(sel), generator=rng).int()
    pool.table.copy_(order[None])
    nats.paged_append(pool, k, v, norm=True, w_k=wk, inv_freq=f)
    pool.check()
    assert torch.equal(ref.slots(pool.k_pages.cpu(), order[None], 0, L, 64), k2[0].cpu())
    tokens = [0, 1, 63, 64, 100, 128, 191, 200, L - 1]
    table, lens = torch.full((len(tokens), len(sel)), -1, dtype=torch.int32), []
    for i, t in enumerate(tokens):
        chunks = [c for c in range(t // 64) if sel[c] == 0] + [t // 64]
        table[i, :len(chunks)] = order[chunks]
        lens.append(64 * (len(chunks) - 1) + t % 64 + 1)
    c = nats.PagedCache(pool.k_pages, pool.v_pages, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    out, lse = nats.paged_decode(c, q2[0, :, tokens].transpose(0, 1).contiguous(), scale=1.0, return_lse=True)
    want = layer["o_soft"][0, :, tokens].transpose(0, 1)
    assert (out.float() - want).abs().max() <= 1e-2 * want.abs().max()
    assert (lse - layer["lse"][0, :, tokens].T).abs().max() <= 1.5e-2


def test_shared_pages_at_uneven_places(nats):
    """Sequences over the same pages whose tiles fall differently among the CTAs: each within the bound, and a call
    repeats bit for bit."""
    rng = torch.Generator().manual_seed(2)
    n, Hk, d, page, B = 5000, 2, 128, 64, 3
    pages = -(-n // page)
    k, v = (torch.randn(pages, Hk, page, d, generator=rng).to(BF) for _ in range(2))
    table = torch.randperm(pages, generator=rng).int()[None]
    q = torch.randn(1, 8, d, generator=rng).to(BF)
    c = nats.PagedCache(k.cuda(), v.cuda(), table.repeat(B, 1).cuda(), torch.full((B,), n, dtype=torch.int32).cuda())
    a, b = (nats.paged_decode(c, q.repeat(B, 1, 1).cuda()) for _ in range(2))
    assert torch.equal(a, b)
    e, _, _, err, _ = ref.decode(q, k, v, table, [n])
    assert ((a.cpu().double() - e).abs() <= 2.0 ** -8 * (e.abs() + err) + err).all()
