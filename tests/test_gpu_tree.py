"""Drafted-token operators (ic_index_score_tree, ic_index_fp_tree,
ic_tree_attn) against their 64-bit forms: sizes, masks, lengths, padding,
refusals, streams and graphs, and one whole step.  Bounds from
tests/tree_ref.py."""
import math

import pytest
import torch

import tests.tree_ref as ref
from cross_layer_top_b200 import synth

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


def trees(B, T, g):
    """Random trees: bit u of mask[b, t] set for t's ancestors and t itself (int64 bits)."""
    mask = torch.zeros((B, T), dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            m = 1 << t
            if t:
                p = int(torch.randint(-1, t, (1,), generator=g))
                if p >= 0:
                    m |= int(mask[b, p]) & (2 ** 64 - 1)
            mask[b, t] = m - (1 << 64) if m >> 63 else m
    return mask


def cu(t):
    return None if t is None else t.cuda()


# ------------------------------------------------------------------- scores
def score_inputs(B, T, H, S, g, integer=False):
    if integer:
        q = torch.randint(-3, 4, (B, T, H, 128), generator=g).bfloat16()
        w = torch.tensor([-1.0, -0.5, 0.5, 1.0])[torch.randint(0, 4, (B, T, H), generator=g)].bfloat16()
        k8 = torch.randint(-4, 5, (B, S, 128), generator=g).float().to(torch.float8_e4m3fn)
        scale = torch.tensor([0.25, 1.0, 2.0])[torch.randint(0, 3, (B, S), generator=g)]
        return q, w, k8.view(torch.uint8), scale
    q = torch.randn((B, T, H, 128), generator=g).bfloat16()
    w = (torch.randn((B, T, H), generator=g) / 8).bfloat16()
    k8, scale = synth.fp8_e4m3_quantize_per_token(torch.randn((B, S, 128), generator=g))
    return q, w, k8.contiguous(), scale.contiguous()


SCORE_CASES = [
    # B, T, H_I, S_max, prefix lengths, draft lengths (None: T each), mask kind
    (1, 1, 64, 1, [0], None, "none"),
    (1, 1, 64, 130, [127], None, "tree"),
    (1, 2, 32, 129, [127], None, "tree"),
    (2, 3, 64, 300, [0, 297], [3, 3], "tree"),
    (3, 4, 64, 700, [128, 1, 690], [4, 0, 2], "tree"),
    (2, 5, 32, 520, [507, 256], None, "none"),
    (2, 8, 64, 1030, [1022, 1000], [8, 7], "tree"),
    (1, 9, 64, 400, [250], None, "tree"),
    (2, 17, 32, 600, [333, 583], [17, 16], "tree"),
    (1, 64, 64, 900, [700], None, "tree"),
    (2, 64, 32, 333, [200, 269], [63, 64], "none"),
    (1, 33, 64, 2100, [2000], [32], "zero"),
    (5, 2, 64, 5000, [4000, 5, 0, 4998, 2500], [2, 2, 2, 2, 1], "tree"),
    (40, 1, 64, 260, [(37 * b) % 259 for b in range(40)], None, "tree"),
]


def masks_of(kind, B, T, g):
    if kind == "none":
        return None
    m = trees(B, T, g)
    if kind == "zero":  # rows that see no draft, not even themselves
        m[:, ::2] = 0
    return m


@pytest.mark.parametrize("integer", [False, True])
@pytest.mark.parametrize("B,T,H,S,prefix,draft,kind", SCORE_CASES)
def test_scores(ic, ctx, B, T, H, S, prefix, draft, kind, integer):
    g = torch.Generator().manual_seed(B * 1000 + T)
    q, w, k8, scale = score_inputs(B, T, H, S, g, integer)
    mask = masks_of(kind, B, T, g)
    d = None if draft is None else torch.tensor(draft, dtype=torch.int32)
    ld = (S + 3) // 4 * 4 + 4
    out = torch.full((B * T, ld), 777.0, device="cuda")
    ic.ic_index_score_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(),
                           torch.tensor(prefix, dtype=torch.int32).cuda(), out, draft_len=cu(d),
                           tree_mask=cu(mask))
    ctx.sync_status()
    got = out.cpu().double().view(B, T, ld)
    for b in range(B):
        m = T if draft is None else draft[b]
        n = prefix[b] + m if m else 0
        want, tol = ref.tree_scores(q[b], w[b], k8[b], scale[b], prefix[b], m,
                                    None if mask is None else mask[b])
        x, want, tol = got[b, :m, :n], want[:, :n], tol[:, :n]  # n = 0 without drafts
        hidden = want == -math.inf
        assert torch.equal(x == -math.inf, hidden)
        if integer:
            assert torch.equal(x, want)
        else:
            assert ((x - want)[~hidden].abs() <= tol[~hidden]).all()
        assert (got[b, :m, n:] == 777.0).all() and (got[b, m:] == 777.0).all()


def test_scores_of_hidden_and_absent_slots_may_hold_anything(ic, ctx):
    """NaN scales and keys behind the last draft and in hidden drafts change nothing visible."""
    B, T, H, S = 2, 6, 64, 500
    g = torch.Generator().manual_seed(5)
    q, w, k8, scale = score_inputs(B, T, H, S, g)
    prefix = torch.tensor([200, 490], dtype=torch.int32)
    mask = torch.tensor([[1, 3, 5, 1, 17, 33]] * B)
    draft = torch.tensor([6, 5], dtype=torch.int32)
    outs = []
    for dirty in (False, True):
        if dirty:
            k8, scale = k8.clone(), scale.clone()
            k8[0, 206:], scale[0, 206:] = 0x7F, float("nan")
            k8[0, 203], scale[0, 203] = 0x7F, float("inf")  # draft 3: no row sees it
            k8[1, 495:], scale[1, 495:] = 0xFF, float("nan")
        out = torch.zeros((B * T, S), device="cuda")
        ic.ic_index_score_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(), prefix.cuda(), out,
                               draft_len=draft.cuda(), tree_mask=mask.cuda())
        ctx.sync_status()
        outs.append(out.cpu())
    assert torch.equal(outs[0], outs[1]) and not torch.isnan(outs[1]).any()


# --------------------------------------------------------------- selections
@pytest.mark.parametrize("B,T,H,S,k,prefix,draft,kind", [
    (1, 1, 64, 64, 64, [10], None, "tree"),
    (2, 4, 64, 600, 64, [500, 60], [4, 3], "tree"),
    (2, 4, 32, 600, 64, [61, 62], None, "tree"),  # around k candidates
    (1, 8, 64, 80, 64, [60], None, "zero"),  # fewer visible than k
    (2, 64, 32, 400, 33, [5, 336], [64, 10], "tree"),
    (3, 5, 64, 3000, 2048, [2995, 2045, 100], [5, 5, 0], "tree"),
    (2, 3, 64, 20000, 2048, [19997, 17000], None, "tree"),  # the cluster top-k
])
def test_selections_exact(ic, ctx, B, T, H, S, k, prefix, draft, kind):
    """Integer inputs: the selected slots are those of a full sort, ties to the lower slot."""
    g = torch.Generator().manual_seed(S + T)
    q, w, k8, scale = score_inputs(B, T, H, S, g, True)
    mask = masks_of(kind, B, T, g)
    d = None if draft is None else torch.tensor(draft, dtype=torch.int32)
    idx = torch.full((B * T, k), -9, dtype=torch.int32, device="cuda")
    ic.ic_index_fp_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(),
                        torch.tensor(prefix, dtype=torch.int32).cuda(), k, idx, draft_len=cu(d),
                        tree_mask=cu(mask))
    ctx.sync_status()
    got = idx.cpu().view(B, T, k)
    for b in range(B):
        m = T if draft is None else draft[b]
        assert (got[b, m:] == -1).all()
        want, _ = ref.tree_scores(q[b], w[b], k8[b], scale[b], prefix[b], m,
                                  None if mask is None else mask[b])
        see = torch.cat([torch.ones((m, prefix[b]), dtype=torch.bool),
                         ref.visible(prefix[b], m, None if mask is None else mask[b], m)], 1)
        for t in range(m):
            s = torch.nonzero(see[t])[:, 0]
            order = torch.sort(want[t, s], descending=True, stable=True).indices[:k]
            sel = s[order].sort().values.to(torch.int32)
            assert torch.equal(got[b, t, :sel.numel()], sel)
            assert (got[b, t, sel.numel():] == -1).all()


def test_chain_equals_decode_steps(ic, ctx):
    """A chain of T drafts selects what T decode steps select (integer inputs: bit for bit)."""
    B, T, H, S, k = 3, 4, 64, 2600, 2048
    g = torch.Generator().manual_seed(11)
    q, w, k8, scale = (t.cuda() for t in score_inputs(B, T, H, S, g, True))
    prefix = torch.tensor([2590, 2047, 300], dtype=torch.int32).cuda()
    idx = torch.empty((B * T, k), dtype=torch.int32, device="cuda")
    ic.ic_index_fp_tree(ctx, q, w, k8, scale, prefix, k, idx)
    for t in range(T):
        one = torch.empty((B, k), dtype=torch.int32, device="cuda")
        ic.ic_index_fp_decode(ctx, q[:, t].contiguous(), w[:, t].contiguous(), k8, scale,
                              prefix + t + 1, k, one)
        assert torch.equal(idx.view(B, T, k)[:, t], one)
    ctx.sync_status()


def test_selection_in_chunks_of_sequences(ic):
    """A small scratch limit cuts the batch into chunks; the result is the same."""
    B, T, H, S, k = 7, 3, 32, 900, 100
    g = torch.Generator().manual_seed(12)
    q, w, k8, scale = (t.cuda() for t in score_inputs(B, T, H, S, g, True))
    prefix = torch.tensor([890, 3, 500, 0, 640, 100, 897], dtype=torch.int32).cuda()
    draft = torch.tensor([3, 3, 2, 3, 0, 1, 3], dtype=torch.int32).cuda()
    mask = trees(B, T, g).cuda()
    outs = []
    for limit in (0, 2 * T * (960 + 1) * 4 + 64):
        c = ic.Context(0, limit)
        idx = torch.empty((B * T, k), dtype=torch.int32, device="cuda")
        ic.ic_index_fp_tree(c, q, w, k8, scale, prefix, k, idx, draft_len=draft, tree_mask=mask)
        c.sync_status()
        outs.append(idx)
        c.close()
    assert torch.equal(outs[0], outs[1])
    c = ic.Context(0, 1000)
    with pytest.raises(ic.ICError) as e:
        ic.ic_index_fp_tree(c, q, w, k8, scale, prefix, k, outs[0])
    assert e.value.code == ic.IC_ERR_NOMEM
    c.close()


# ---------------------------------------------------------------- attention
def attn_inputs(B, T, Hq, d, S, g):
    return (torch.randn((B, T, Hq, d), generator=g).bfloat16(),
            torch.randn((B, S, d), generator=g).bfloat16(),
            torch.randn((B, S, d), generator=g).bfloat16())


def lists(B, k, prefix, g, holes=False):
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b in range(B):
        p = torch.randperm(max(prefix[b], 1), generator=g)[:min(k, prefix[b])].sort().values
        idx[b, :p.numel()] = p.to(torch.int32)
    if holes:  # -1 anywhere, any order
        idx[:, ::3] = -1
        idx = idx[:, torch.randperm(k, generator=g)].contiguous()
    return idx


def check_attn(got, Q, K, V, prefix, draft, mask, idx, T, scale, fill):
    for b in range(Q.shape[0]):
        m = T if draft is None else int(draft[b])
        want, tol = ref.tree_attn(Q[b], K[b], V[b], prefix[b], m, None if mask is None else mask[b],
                                  None if idx is None else idx[b], scale)
        err = (got[b, :m].double() - want).abs()
        assert (err <= tol).all(), (b, err.max(), (err / tol.clamp_min(1e-30)).max())
        assert (got[b, m:] == fill).all()


ATTN_CASES = [
    # B, T, Hq, d, S, k (0: whole prefix), prefix, draft, mask kind
    (1, 1, 1, 64, 1, 0, [0], None, "tree"),
    (1, 1, 16, 128, 130, 0, [129], None, "none"),
    (1, 3, 4, 64, 333, 0, [330], None, "tree"),
    (2, 2, 16, 128, 128, 0, [126, 0], None, "tree"),
    (2, 8, 16, 128, 257, 0, [249, 128], [8, 5], "tree"),
    (3, 5, 7, 128, 400, 0, [395, 1, 120], [5, 0, 3], "tree"),
    (1, 9, 16, 64, 1500, 0, [1491], None, "tree"),
    (2, 16, 16, 128, 700, 0, [600, 684], [16, 11], "tree"),
    (1, 17, 16, 128, 513, 0, [300], None, "none"),
    (1, 64, 16, 128, 1000, 0, [936], None, "tree"),
    (2, 64, 16, 64, 777, 0, [713, 64], [64, 33], "tree"),
    (2, 33, 5, 128, 300, 0, [200, 0], [33, 20], "zero"),
    (1, 4, 16, 128, 9000, 0, [8996], None, "tree"),
    (40, 2, 16, 128, 260, 0, [(31 * b) % 258 for b in range(40)], None, "tree"),
    (1, 1, 16, 128, 200, 64, [190], None, "tree"),
    (2, 8, 16, 128, 5000, 2048, [4992, 700], None, "tree"),
    (3, 11, 7, 64, 900, 517, [889, 100, 0], [11, 4, 2], "tree"),
    (2, 64, 16, 128, 3100, 2048, [3000, 2500], [64, 1], "tree"),
    (2, 20, 16, 128, 600, 1, [500, 580], None, "none"),
    (1, 5, 16, 64, 600, 129, [595], None, "zero"),
    (3, 3, 2, 128, 300, 200, [0, 297, 150], [3, 3, 0], "zero"),
    # more (sequence, row group) units than CTAs, some of one key tile: several per CTA
    (500, 2, 8, 64, 140, 0, [(7 * b) % 139 for b in range(500)], None, "tree"),
    (300, 3, 16, 128, 300, 0, [(29 * b) % 298 for b in range(300)], None, "tree"),
    (200, 9, 16, 64, 150, 100, [(13 * b) % 142 for b in range(200)], [b % 10 for b in range(200)], "tree"),
]


@pytest.mark.parametrize("B,T,Hq,d,S,k,prefix,draft,kind", ATTN_CASES)
def test_attention(ic, ctx, B, T, Hq, d, S, k, prefix, draft, kind):
    g = torch.Generator().manual_seed(S * 7 + T)
    Q, K, V = attn_inputs(B, T, Hq, d, S, g)
    mask = masks_of(kind, B, T, g)
    idx = lists(B, k, prefix, g, holes=bool(T & 1)) if k else None
    dl = None if draft is None else torch.tensor(draft, dtype=torch.int32)
    out = torch.full((B, T, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(),
                    torch.tensor(prefix, dtype=torch.int32).cuda(), out, idx=cu(idx),
                    draft_len=cu(dl), tree_mask=cu(mask))
    ctx.sync_status()
    check_attn(out.cpu(), Q, K, V, prefix, draft, mask, idx, T, 1 / math.sqrt(d), 3.0)


@pytest.mark.parametrize("k", [0, 600])
@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_attention_peaked_and_flat(ic, ctx, k, size):
    """Near-uniform weights, and logits hundreds apart that move the running maximum."""
    B, T, Hq, d, S = 2, 6, 16, 128, 1400
    g = torch.Generator().manual_seed(21)
    Q, K, V = attn_inputs(B, T, Hq, d, S, g)
    Q = (Q.float() * size).bfloat16()
    ramp = torch.linspace(0.1, 1.0, S)[None, :, None]  # later keys are larger
    K = (K.float() * ramp).bfloat16()
    prefix = [1394, 900]
    mask = trees(B, T, g)
    idx = lists(B, k, prefix, g) if k else None
    out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(),
                    torch.tensor(prefix, dtype=torch.int32).cuda(), out, idx=cu(idx),
                    tree_mask=mask.cuda(), scale=0.05)
    ctx.sync_status()
    check_attn(out.cpu(), Q, K, V, prefix, None, mask, idx, T, 0.05, 0.0)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_ignores_what_no_row_sees(ic, ctx, d):
    """NaN and infinities behind the last draft, in slots off the list and in drafts that no row
    sees leave every output as it was; the same for a cache's next sequence."""
    B, T, Hq, S, k = 2, 6, 8, 700, 300
    g = torch.Generator().manual_seed(31)
    Q, K, V = attn_inputs(B, T, Hq, d, S, g)
    prefix, draft = [500, 690], [6, 5]
    mask = torch.tensor([[1, 3, 5, 1, 17, 33]] * B)  # no row sees draft 3
    for idx in (None, lists(B, k, prefix, g)):
        outs = []
        for dirty in (False, True):
            K2, V2 = K.clone(), V.clone()
            if dirty:
                for b in range(B):
                    gone = torch.ones(S, dtype=torch.bool)
                    gone[:prefix[b]] = False
                    if idx is not None:
                        gone[:prefix[b]] = True
                        gone[idx[b][idx[b] >= 0].long()] = False
                    for u in (0, 1, 2, 4, 5):
                        if u < draft[b]:
                            gone[prefix[b] + u] = False
                    K2[b, gone], V2[b, gone] = float("nan"), float("inf")
            out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
            ic.ic_tree_attn(ctx, Q.cuda(), K2.cuda(), V2.cuda(),
                            torch.tensor(prefix, dtype=torch.int32).cuda(), out, idx=cu(idx),
                            draft_len=torch.tensor(draft, dtype=torch.int32).cuda(),
                            tree_mask=mask.cuda())
            ctx.sync_status()
            outs.append(out.cpu())
        assert torch.equal(outs[0], outs[1])


def test_attention_repeated_listed_positions_count_twice(ic, ctx):
    B, T, Hq, d, S = 1, 2, 4, 64, 100
    g = torch.Generator().manual_seed(41)
    Q, K, V = attn_inputs(B, T, Hq, d, S, g)
    idx = torch.tensor([[5, 5, 5, 90, -1, 17]], dtype=torch.int32)
    out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(), torch.tensor([95], dtype=torch.int32).cuda(),
                    out, idx=idx.cuda())
    ctx.sync_status()
    check_attn(out.cpu(), Q, K, V, [95], None, None, idx, T, 0.125, 0.0)


@pytest.mark.parametrize("k", [0, 200])
def test_attention_on_interleaved_caches(ic, ctx, k):
    """K and V as halves of one [B, 2, S, d] cache: sequences two caches apart."""
    B, T, Hq, d, S = 3, 4, 16, 128, 700
    g = torch.Generator().manual_seed(43)
    Q, K, V = attn_inputs(B, T, Hq, d, S, g)
    kv = torch.stack([K, V], 1).cuda()
    prefix, mask = [696, 300, 5], trees(B, T, g)
    idx = lists(B, k, prefix, g) if k else None
    out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), kv[:, 0], kv[:, 1], torch.tensor(prefix, dtype=torch.int32).cuda(),
                    out, idx=cu(idx), tree_mask=mask.cuda())
    ctx.sync_status()
    check_attn(out.cpu(), Q, K, V, prefix, None, mask, idx, T, d ** -0.5, 0.0)


# ------------------------------------------------------- errors and refusals
def test_bad_lengths_and_indices_are_reported(ic, ctx):
    B, T, S = 3, 4, 64
    g = torch.Generator().manual_seed(51)
    Q, K, V = (t.cuda() for t in attn_inputs(B, T, 4, 64, S, g))
    q, w, k8, scale = (t.cuda() for t in score_inputs(B, T, 32, S, g))
    good = [30, 60, 10]
    for at, prefix, draft in [(1, 61, 4), (1, -1, 4), (1, 5, 5), (1, 5, -1), (2, 2 ** 31 - 1, 4)]:
        p = torch.tensor(good, dtype=torch.int32)
        dl = torch.full((B,), T, dtype=torch.int32)
        p[at], dl[at] = prefix, draft
        out = torch.full((B, T, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        ic.ic_tree_attn(ctx, Q, K, V, p.cuda(), out, draft_len=dl.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE and "prefix_len" in str(e.value)
        same = (out == 3.0).flatten(1).all(1).cpu()
        assert same[at] and same.sum() == 1
        sc = torch.full((B * T, S), 3.0, device="cuda")
        ic.ic_index_score_tree(ctx, q, w, k8, scale, p.cuda(), sc, draft_len=dl.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE
        same = (sc.view(B, -1) == 3.0).all(1).cpu()
        assert same[at] and same.sum() == 1
        idx = torch.full((B * T, 8), -9, dtype=torch.int32, device="cuda")
        ic.ic_index_fp_tree(ctx, q, w, k8, scale, p.cuda(), 8, idx, draft_len=dl.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE
        assert ((idx.view(B, -1) == -1).all(1).cpu() == torch.arange(B).eq(at)).all()
    # indices outside the committed slots, drafts among them, are skipped
    idx = lists(B, 9, good, g)
    want = torch.zeros((B, T, 4, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor(good, dtype=torch.int32).cuda()
    clean = idx.clone()
    clean[1, 4] = -1
    ic.ic_tree_attn(ctx, Q, K, V, pos, want, idx=clean.cuda())
    ctx.sync_status()
    for bad in (-2, 60, 63, 2 ** 31 - 1):
        idx[1, 4] = bad
        out = torch.zeros_like(want)
        ic.ic_tree_attn(ctx, Q, K, V, pos, out, idx=idx.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE
        assert torch.equal(out, want)
    ctx.sync_status()


def test_refusals(ic, ctx):
    B, T, S = 2, 4, 64
    g = torch.Generator().manual_seed(61)
    Q, K, V = (t.cuda() for t in attn_inputs(B, T, 4, 64, S, g))
    q, w, k8, scale = (t.cuda() for t in score_inputs(B, T, 32, S, g))
    p = torch.full((B,), 10, dtype=torch.int32, device="cuda")
    out = torch.empty_like(Q)
    sc = torch.empty((B * T, S), device="cuda")
    idx = torch.zeros((B, 8), dtype=torch.int32, device="cuda")

    def code(f, *a, **kw):
        with pytest.raises(ic.ICError) as e:
            f(ctx, *a, **kw)
        return e.value.code

    big = torch.zeros((B, 65, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert code(ic.ic_tree_attn, big, K, V, p, torch.empty_like(big)) == ic.IC_ERR_UNSUPPORTED
    wide = torch.zeros((B, T, 17, 64), dtype=torch.bfloat16, device="cuda")
    assert code(ic.ic_tree_attn, wide, K, V, p, torch.empty_like(wide)) == ic.IC_ERR_SHAPE
    thin = torch.zeros((B, T, 4, 32), dtype=torch.bfloat16, device="cuda")
    assert code(ic.ic_tree_attn, thin, K[..., :32].contiguous(), V[..., :32].contiguous(), p,
                torch.empty_like(thin)) == ic.IC_ERR_UNSUPPORTED
    many = torch.zeros((B, 2049), dtype=torch.int32, device="cuda")
    assert code(ic.ic_tree_attn, Q, K, V, p, out, idx=many) == ic.IC_ERR_SHAPE
    skew = torch.zeros(Q.numel() + 4, dtype=torch.bfloat16, device="cuda")[4:].view(Q.shape)
    assert code(ic.ic_tree_attn, skew, K, V, p, out) == ic.IC_ERR_INVALID_ARG
    # the output on an input
    assert code(ic.ic_tree_attn, Q, K, V, p, Q) == ic.IC_ERR_INVALID_ARG
    if B * T * 4 <= K.shape[0] * K.shape[1]:
        assert code(ic.ic_tree_attn, Q, K, V, p, V.view(-1)[:Q.numel()].view(Q.shape)) == ic.IC_ERR_INVALID_ARG
    for bad in (lambda: ic.ic_tree_attn(ctx, Q.cpu(), K, V, p, out),
                lambda: ic.ic_tree_attn(ctx, Q, K, V[:, :-1].contiguous(), p, out),
                lambda: ic.ic_tree_attn(ctx, Q, K, V, p[:1], out),
                lambda: ic.ic_tree_attn(ctx, Q, K, V, p.long(), out),
                lambda: ic.ic_tree_attn(ctx, Q, K, V, p, out, idx=idx[:1]),
                lambda: ic.ic_tree_attn(ctx, Q, K.transpose(1, 2), V, p, out),
                lambda: ic.ic_tree_attn(ctx, Q, torch.cat([K, K], 2)[..., :64], V, p, out),
                lambda: ic.ic_tree_attn(ctx, Q, K, V, p, out, idx=idx[:, :0].contiguous()),
                lambda: ic.ic_index_score_tree(ctx, q, w[:1], k8, scale, p, sc),
                lambda: ic.ic_index_score_tree(ctx, q, w, k8, scale, p, sc[:3])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    assert code(ic.ic_index_score_tree, q, w, k8, scale, p, sc[:, :60].contiguous()) == ic.IC_ERR_SHAPE
    q16 = torch.zeros((B, T, 16, 128), dtype=torch.bfloat16, device="cuda")
    w16 = torch.zeros((B, T, 16), dtype=torch.bfloat16, device="cuda")
    assert code(ic.ic_index_score_tree, q16, w16, k8, scale, p, sc) == ic.IC_ERR_UNSUPPORTED
    q65 = torch.zeros((B, 65, 32, 128), dtype=torch.bfloat16, device="cuda")
    w65 = torch.zeros((B, 65, 32), dtype=torch.bfloat16, device="cuda")
    assert code(ic.ic_index_score_tree, q65, w65, k8, scale, p,
                torch.empty((B * 65, S), device="cuda")) == ic.IC_ERR_UNSUPPORTED
    o = torch.empty((B * T, 2049), dtype=torch.int32, device="cuda")
    assert code(ic.ic_index_fp_tree, q, w, k8, scale, p, 2049, o) == ic.IC_ERR_SHAPE
    ctx.sync_status()


# ------------------------------------------------------- streams and graphs
def test_captured_and_replayed_on_new_contents(ic):
    """Scores, selections and attention in one captured graph, on a stream of its own, replayed
    with other lengths, trees and keys; the context's first calls come before the capture."""
    ctx = ic.Context(0)
    B, T, H, S, k, Hq, d = 3, 5, 64, 3000, 256, 16, 128
    bufs = None
    graph = None
    s = torch.cuda.Stream()
    for seed in range(3):
        g = torch.Generator().manual_seed(70 + seed)
        new = list(score_inputs(B, T, H, S, g, True)) + list(attn_inputs(B, T, Hq, d, S, g))
        new += [torch.randint(0, S - T, (B,), generator=g, dtype=torch.int32),
                torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32), trees(B, T, g)]
        if bufs is None:
            bufs = [t.cuda() for t in new]
            idx = torch.zeros((B * T, k), dtype=torch.int32, device="cuda")
            out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
            out2, out3 = torch.zeros_like(out), torch.zeros_like(out)
        else:
            for a, b in zip(bufs, new):
                a.copy_(b)
        q, w, k8, scale, Q, K, V, prefix, draft, mask = bufs

        def step():
            ic.ic_index_fp_tree(ctx, q, w, k8, scale, prefix, k, idx, draft_len=draft, tree_mask=mask)
            ic.ic_sparse_attn(ctx, Q.view(B * T, Hq, d), K, V, idx, out, rows_per_seq=T,
                              kv_seq_stride=S * d)
            ic.ic_tree_attn(ctx, Q, K, V, prefix, out2, draft_len=draft, tree_mask=mask)
            ic.ic_tree_attn(ctx, Q, K, V, prefix, out3, idx=sel, draft_len=draft, tree_mask=mask)

        if graph is None:
            sel = torch.full((B, 17), -1, dtype=torch.int32, device="cuda")
            sel[:, :2] = torch.tensor([0, 1])
            prefix.clamp_(min=2)
            step()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        prefix.clamp_(min=2)
        for o in (idx, out, out2, out3):
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (idx, out, out2, out3)]
        for o in (idx, out, out2, out3):
            o.zero_()
        step()
        ctx.sync_status()
        for a, b in zip(got, (idx, out, out2, out3)):
            assert torch.equal(a, b)
        check_attn(got[2].cpu(), Q.cpu(), K.cpu(), V.cpu(), prefix.tolist(), draft.tolist(),
                   mask.cpu(), None, T, d ** -0.5, 0.0)
    del graph
    ctx.close()


def test_first_calls_inside_a_capture_are_refused(ic):
    """A first call that would have to allocate says so and leaves the capture alive; a captured
    call's scratch does not move afterwards."""
    ctx = ic.Context(0)
    B, T, H, S, k = 2, 3, 32, 500, 64
    g = torch.Generator().manual_seed(83)
    q, w, k8, scale = (t.cuda() for t in score_inputs(B, T, H, S, g, True))
    Q, K, V = (t.cuda() for t in attn_inputs(B, T, 4, 64, S, g))
    prefix = torch.tensor([490, 100], dtype=torch.int32).cuda()
    idx = torch.zeros((B * T, k), dtype=torch.int32, device="cuda")
    out = torch.zeros_like(Q)

    def calls():
        ic.ic_index_fp_tree(ctx, q, w, k8, scale, prefix, k, idx)
        ic.ic_tree_attn(ctx, Q, K, V, prefix, out)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out.fill_(1.0)
        for f in (lambda: ic.ic_index_fp_tree(ctx, q, w, k8, scale, prefix, k, idx),
                  lambda: ic.ic_tree_attn(ctx, Q, K, V, prefix, out)):
            with pytest.raises(ic.ICError) as e:
                f()
            assert e.value.code == ic.IC_ERR_NOMEM and "capture" in str(e.value)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 1.0).all()
    calls()
    ctx.sync_status()
    want = idx.clone(), out.clone()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2, stream=s):
        calls()
    big = score_inputs(B, T, H, 5 * S, g, True)
    with pytest.raises(ic.ICError) as e:
        ic.ic_index_fp_tree(ctx, q, w, big[2].cuda(), big[3].cuda(), prefix, k, idx)
    assert e.value.code == ic.IC_ERR_NOMEM and "captured" in str(e.value)
    idx.zero_()
    out.zero_()
    graph2.replay()
    ctx.sync_status()
    assert torch.equal(idx, want[0]) and torch.equal(out, want[1])
    del graph, graph2
    ctx.close()


def test_two_contexts_on_two_streams(ic):
    """Calls of two contexts in flight at once do not touch each other's workspaces."""
    B, T, Hq, d, S = 2, 8, 16, 128, 20000
    g = torch.Generator().manual_seed(81)
    ctxs = [ic.Context(0) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    data = [[t.cuda() for t in attn_inputs(B, T, Hq, d, S, g)] for _ in range(2)]
    prefix = torch.tensor([S - T, S - T - 77], dtype=torch.int32).cuda()
    want = []
    for i in range(2):
        o = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
        ic.ic_tree_attn(ctxs[i], *data[i], prefix, o)
        ctxs[i].sync_status()
        want.append(o)
    outs = [[torch.zeros_like(want[0]) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for j in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ic.ic_tree_attn(ctxs[i], *data[i], prefix, outs[i][j])
    for i in range(2):
        ctxs[i].sync_status(streams[i])
        assert all(torch.equal(o, want[i]) for o in outs[i])
        ctxs[i].close()


# ------------------------------------------------------------- a whole step
def test_a_drafted_step(ic, ctx):
    """Projected rows -> norms, rotations and cache writes -> each draft's own selection and its
    sparse attention, and the tree attention over the whole prefix and over the root's list."""
    B, T, S, k, Hq, d, H = 3, 6, 2500, 512, 16, 128, 64
    g = torch.Generator().manual_seed(91)
    prefix = torch.tensor([2400, 600, 2494], dtype=torch.int32)
    mask = trees(B, T, g)
    depth = torch.tensor([[bin(int(v) & (2 ** 64 - 1)).count("1") - 1 for v in r] for r in mask])
    pos = (prefix[:, None] + depth).to(torch.int32).flatten()
    slot = (torch.arange(B)[:, None] * S + prefix[:, None] + torch.arange(T)).flatten().long()
    f = torch.cat([torch.ones(d // 2), torch.zeros(d // 2)])
    ang = torch.arange(4096, dtype=torch.float64)[:, None] * (
        10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d))
    rope = torch.cat([ang.cos(), ang.sin()], 1).float()
    ropeI = torch.cat([ang[:, ::2].cos(), ang[:, ::2].sin()], 1).float()
    assert rope[0].equal(f)
    rows = B * T
    qkv = torch.randn((rows, (Hq + 2) * d), generator=g).bfloat16()
    iqk = torch.randn((rows, (H + 1) * d), generator=g).bfloat16()
    wq, wk, wi, bi = (1 + 0.1 * torch.randn(d, generator=g) for _ in range(4))
    K, V = (torch.randn((B, S, d), generator=g).bfloat16().cuda() for _ in range(2))
    k8, sc = synth.fp8_e4m3_quantize_per_token(torch.randn((B, S, d), generator=g))
    k8, sc = k8.contiguous().cuda(), sc.contiguous().cuda()
    w = (torch.randn((B, T, H), generator=g) / 8).bfloat16()
    Q = torch.empty((rows, Hq, d), dtype=torch.bfloat16, device="cuda")
    qI = torch.empty((rows, H, d), dtype=torch.bfloat16, device="cuda")
    a, b = qkv.cuda(), iqk.cuda()
    sl = slot.cuda()
    ic.ic_qk_norm_rope(ctx, [
        dict(x=a[:, :Hq * d].unflatten(1, (Hq, d)), norm="rms", weight=wq.cuda(), rope=rope.cuda(), out=Q),
        dict(x=a[:, Hq * d:(Hq + 1) * d].unflatten(1, (1, d)), norm="rms", weight=wk.cuda(),
             rope=rope.cuda(), out=K, slot=sl),
        dict(x=a[:, (Hq + 1) * d:].unflatten(1, (1, d)), out=V, slot=sl),
        dict(x=b[:, :H * d].unflatten(1, (H, d)), rope=ropeI.cuda(), out=qI),
        dict(x=b[:, H * d:].unflatten(1, (1, d)), norm="layer", weight=wi.cuda(), bias=bi.cuda(),
             rope=ropeI.cuda(), out8=k8, out_scale=sc, slot=sl)], pos.cuda())
    # what the first call made, against its formula
    x = qkv.unflatten(1, (Hq + 2, d))
    z, tol = ref.norm_rope(x[:, :Hq], "rms", wq, None, 1e-6, rope, pos, False)
    assert ((Q.cpu().double() - z).abs() <= tol + (z.abs() + tol) * ref.UBF16).all()
    z, tol = ref.norm_rope(x[:, Hq:Hq + 1], "rms", wk, None, 1e-6, rope, pos, False)
    Kc = K.cpu()
    assert ((Kc.view(B * S, d)[slot].double() - z[:, 0]).abs() <=
            tol[:, 0] + (z[:, 0].abs() + tol[:, 0]) * ref.UBF16).all()
    Vc = V.cpu()
    assert torch.equal(Vc.view(B * S, d)[slot], x[:, Hq + 1])
    # each draft's own selection, and attention at it
    idx = torch.empty((rows, k), dtype=torch.int32, device="cuda")
    q4 = qI.view(B, T, H, d)
    ic.ic_index_fp_tree(ctx, q4, w.cuda(), k8, sc, prefix.cuda(), k, idx, tree_mask=mask.cuda())
    own = torch.empty((rows, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_sparse_attn(ctx, Q, K, V, idx, own, rows_per_seq=T, kv_seq_stride=S * d)
    # the whole prefix, and the list that the root selected of it
    root = idx.view(B, T, k)[:, 0].clone()
    root[root >= prefix.cuda()[:, None]] = -1
    whole, shared = (torch.empty((B, T, Hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q4 = Q.view(B, T, Hq, d)
    ic.ic_tree_attn(ctx, Q4, K, V, prefix.cuda(), whole, tree_mask=mask.cuda())
    ic.ic_tree_attn(ctx, Q4, K, V, prefix.cuda(), shared, idx=root, tree_mask=mask.cuda())
    ctx.sync_status()
    got = idx.cpu().view(B, T, k)
    for b_ in range(B):
        s, tol = ref.tree_scores(q4[b_].cpu(), w[b_], k8[b_].cpu(), sc[b_].cpu(), int(prefix[b_]), T, mask[b_])
        for t in range(T):
            sel = got[b_, t][got[b_, t] >= 0].long()
            n = int((s[t] > -math.inf).sum())
            assert sel.numel() == min(k, n) and (sel.diff() > 0).all()
            kth = s[t].topk(sel.numel()).values[-1]
            assert (s[t, sel] >= kth - 2 * tol[t].max()).all()
            # sparse attention at exactly those slots
            o, tl = attend(Q4[b_, t].cpu(), Kc[b_], Vc[b_], sel, d ** -0.5)
            assert ((own.view(B, T, Hq, d)[b_, t].cpu().double() - o).abs() <= tl).all()
    check_attn(whole.cpu(), Q4.cpu(), Kc, Vc, prefix.tolist(), None, mask, None, T, d ** -0.5, 0.0)
    check_attn(shared.cpu(), Q4.cpu(), Kc, Vc, prefix.tolist(), None, mask, root.cpu(), T, d ** -0.5, 0.0)


def attend(q, K, V, sel, scale):
    """Attention of one row's heads at the slots `sel`, with the same bound."""
    Ks, Vs = K[sel], V[sel]
    n = sel.numel()
    out, tol = ref.tree_attn(q[None], torch.cat([Ks, Ks[:1]]), torch.cat([Vs, Vs[:1]]), n, 1,
                             torch.zeros(1, dtype=torch.int64), None, scale)
    return out[0], tol[0]
