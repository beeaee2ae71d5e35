"""Drafted-token attention with NaN and infinities in queries and keys: they
stay in the rows that meet them, and those are what the formula gives.  And
selections of more rows than the cluster top-k takes."""
import math

import pytest
import torch

import tests.tree_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ic():
    from cross_layer_top_b200 import indexcache
    return indexcache


@pytest.fixture(scope="module")
def ctx(ic):
    c = ic.Context(0)
    yield c
    c.close()


def run(ic, ctx, Q, K, V, prefix, mask=None, idx=None, draft=None):
    out = torch.full(Q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(), torch.tensor(prefix, dtype=torch.int32).cuda(), out,
                    idx=cu(idx), draft_len=cu(draft), tree_mask=cu(mask))
    ctx.sync_status()
    return out.cpu()


@pytest.mark.parametrize("T,S", [(4, 700), (20, 700), (4, 40000), (20, 40000)])
def test_not_a_number_in_a_query_stays_in_its_row(ic, ctx, T, S):
    B, Hq, d = 2, 16, 128
    g = torch.Generator().manual_seed(T)
    Q = torch.randn((B, T, Hq, d), generator=g).bfloat16()
    K, V = (torch.randn((B, S, d), generator=g).bfloat16() for _ in range(2))
    prefix = [S - T, S // 2]
    clean = run(ic, ctx, Q, K, V, prefix)
    Q[0, 1, 3, 17] = math.nan
    Q[1, T - 1, 0, 0] = math.nan
    got = run(ic, ctx, Q, K, V, prefix)
    bad = torch.zeros((B, T, Hq), dtype=torch.bool)
    bad[0, 1, 3] = bad[1, T - 1, 0] = True
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], clean[~bad])


def test_padding_queries_may_hold_anything(ic, ctx):
    B, T, Hq, d, S = 2, 12, 16, 64, 900
    g = torch.Generator().manual_seed(8)
    Q = torch.randn((B, T, Hq, d), generator=g).bfloat16()
    K, V = (torch.randn((B, S, d), generator=g).bfloat16() for _ in range(2))
    draft = torch.tensor([5, 0], dtype=torch.int32)
    clean = run(ic, ctx, Q, K, V, [800, 700], draft=draft)
    Q[0, 5:], Q[1] = math.nan, math.inf
    got = run(ic, ctx, Q, K, V, [800, 700], draft=draft)
    assert torch.equal(got, clean) and (got[0, 5:] == 3.0).all() and (got[1] == 3.0).all()


@pytest.mark.parametrize("S", [300, 40000])
def test_keys_of_infinite_logits(ic, ctx, S):
    """A logit of -inf has weight 0 wherever it stands; a row whose every logit is -inf sees nothing
    and is zero."""
    B, T, Hq, d = 1, 3, 4, 64
    g = torch.Generator().manual_seed(S)
    Q = torch.randn((B, T, Hq, d), generator=g).bfloat16()
    Q[..., 0] = Q[..., 0].abs() + 0.5
    Q[0, 1, 2] = 0
    Q[0, 1, 2, 0] = 1.0
    K, V = (torch.randn((B, S, d), generator=g).bfloat16() for _ in range(2))
    n = S - T
    K[:, :n:2, 0] = -math.inf  # every second committed key
    got = run(ic, ctx, Q, K, V, [n])
    kept = torch.cat([torch.arange(1, n, 2), n + torch.arange(T)])
    want, tol = ref.tree_attn(Q[0], K[0, kept], V[0, kept], kept.numel() - T, T, None, None, d ** -0.5)
    assert ((got[0].double() - want).abs() <= tol).all()
    K[..., 0] = -math.inf
    assert (run(ic, ctx, Q, K, V, [n]) == 0).all()


def test_selections_of_many_long_rows(ic, ctx):
    """80 rows, which the cluster top-k does not take; ties everywhere."""
    B, T, H, S, k = 20, 4, 64, 20011, 2048
    g = torch.Generator().manual_seed(5)
    q = torch.randint(-1, 2, (B, T, H, 128), generator=g).bfloat16()
    w = torch.tensor([-0.5, 0.5])[torch.randint(0, 2, (B, T, H), generator=g)].bfloat16()
    k8 = torch.randint(-1, 2, (B, S, 128), generator=g).float().to(torch.float8_e4m3fn)
    scale = torch.ones((B, S))
    prefix = torch.randint(k, S - T, (B,), generator=g, dtype=torch.int32)
    prefix[0], prefix[1], prefix[2] = S - T, 17, 2047
    draft = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    draft[:3] = T
    mask = torch.tensor([1, 3, 5, 0]).expand(B, T).contiguous()
    idx = torch.full((B * T, k), -9, dtype=torch.int32, device="cuda")
    ic.ic_index_fp_tree(ctx, q.cuda(), w.cuda(), k8.view(torch.uint8).cuda(), scale.cuda(), prefix.cuda(), k, idx,
                        draft_len=draft.cuda(), tree_mask=mask.cuda())
    ctx.sync_status()
    got = idx.view(B, T, k)
    for b in range(B):
        n, m = int(prefix[b]), int(draft[b])
        assert (got[b, m:] == -1).all()
        keys = k8[b, :n + m].cuda().double()
        see = torch.cat([torch.ones((m, n), dtype=torch.bool), ref.visible(n, m, mask[b], m)], 1).cuda()
        for t in range(m):
            score = w[b, t].cuda().double() @ (q[b, t].cuda().double() @ keys.T).clamp_min(0)
            s = torch.nonzero(see[t])[:, 0]
            order = torch.sort(score[s], descending=True, stable=True).indices[:k]
            sel = s[order].sort().values.int()
            assert torch.equal(got[b, t, :sel.numel()], sel) and (got[b, t, sel.numel():] == -1).all()
