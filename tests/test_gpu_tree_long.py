"""Drafted-token operators where a CTA has many key tiles of a part, or several
parts one after another: rings that go round, barrier phases past the first,
accumulators carried from part to part, and a running maximum that moves.
How many tiles a CTA gets is worked out here as the kernels do, so that a case
cannot lose what it is for."""
import math

import pytest
import torch

import tests.tree_ref as ref

pytestmark = pytest.mark.gpu

TILE = 128  # keys


@pytest.fixture(scope="module")
def ic():
    from cross_layer_top_b200 import indexcache
    return indexcache


@pytest.fixture(scope="module")
def ctx(ic):
    c = ic.Context(0)
    yield c
    c.close()


def parts_of(units, slack):
    """Per CTA, the key tiles of each of its parts.  units: key tiles of each (sequence, row group), in
    order.  Cut into equal pieces of at most mean + s tiles, with the least s in 0..slack that gives no
    more pieces than CTAs; else into equal ranges of the line."""
    ctas, total = torch.cuda.get_device_properties(0).multi_processor_count, sum(units)
    mean = -(-total // ctas)
    for step in range(mean, mean + slack + 1):
        cuts = [-(-t // step) for t in units]
        if sum(cuts) <= ctas:
            return [[t * (i + 1) // n - t * i // n] for t, n in zip(units, cuts) for i in range(n)]
    n = min(total, ctas)
    out, at, begin = [], 0, 0
    ends = []
    for t in units:
        at += t
        ends.append(at)
    for c in range(n):
        end = total * (c + 1) // n
        mine = []
        while begin < end:
            stop = min(end, next(e for e in ends if e > begin))
            mine.append(stop - begin)
            begin = stop
        out.append(mine)
    return out


def units_of(lens, drafts, rows_per_draft, group_rows):
    return [-(-(n + m) // TILE) for n, m in zip(lens, drafts)
            for _ in range(-(-m * rows_per_draft // group_rows))]


def chains(B, T):
    """Masks of trees whose node t hangs from node (t - 1) // 2, as int64 bits."""
    m = torch.zeros((B, T), dtype=torch.int64)
    for t in range(T):
        bits = 1 << t
        if t:
            bits |= int(m[0, (t - 1) // 2]) & (2 ** 64 - 1)
        m[:, t] = bits - (1 << 64) if bits >> 63 else bits
    return m


# ------------------------------------------------------------------ attention
def attend(q, K, V, sel, scale):
    """One query row's heads at the slots `sel`: the 64-bit form, its bound and the logits."""
    n = sel.numel()
    out, tol = ref.tree_attn(q[None], torch.cat([K[sel], K[:1]]), torch.cat([V[sel], V[:1]]), n, 1,
                             torch.zeros(1, dtype=torch.int64), None, scale)
    return out[0], tol[0]


@pytest.mark.parametrize("B,T,d,S,k", [(4, 8, 128, 40007, 0), (4, 8, 64, 39999, 0), (4, 5, 128, 39000, 0),
                                       (4, 64, 128, 15990, 0), (4, 64, 64, 16001, 0), (150, 8, 128, 3001, 2048),
                                       (40, 64, 64, 3001, 2048)])
def test_attention_over_many_tiles(ic, ctx, B, T, d, S, k):
    """The keys grow tenfold every eight tiles, so a row's maximum passes its reference by far more
    than 2^8 several times in a part, and O, of the tiles before, is scaled down in TMEM."""
    Hq, scale = 16, 0.05
    g = torch.Generator().manual_seed(T + d)
    prefix = [S - T - 131 * (b % 7) for b in range(B)]
    wide = T * Hq > 128  # two row tiles a CTA
    units = units_of([k] * B if k else prefix, [T] * B, Hq, 256 if wide else 128)
    assert min(max(p) for p in parts_of(units, 2 if wide else 4)) >= 4
    Q = (torch.randn((B, T, Hq, d), generator=g) * 20).bfloat16()
    grow = 0.1 + 0.9 * ((torch.arange(S) // TILE) % 8) / 7
    K = (torch.randn((B, S, d), generator=g) * grow[None, :, None]).bfloat16()
    V = torch.randn((B, S, d), generator=g).bfloat16()
    idx = None
    if k:
        idx = torch.full((B, k), -1, dtype=torch.int32)
        for b in range(B):
            p = torch.randperm(prefix[b], generator=g)[:k].sort().values
            idx[b, :p.numel()] = p.to(torch.int32)
    mask = chains(B, T)
    out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(), torch.tensor(prefix, dtype=torch.int32).cuda(), out,
                    idx=None if idx is None else idx.cuda(), tree_mask=mask.cuda(), scale=scale)
    ctx.sync_status()
    got = out.cpu().double()
    moved = 0
    for b in range(0, B, max(1, B // 8)):
        for t in (0, T // 2, T - 1):
            seen = torch.tensor([u for u in range(T) if int(mask[b, t]) >> u & 1])
            base = torch.arange(prefix[b]) if idx is None else idx[b][idx[b] >= 0].long()
            sel = torch.cat([base, prefix[b] + seen])
            want, tol = attend(Q[b, t], K[b], V[b], sel, scale)
            err = (got[b, t] - want).abs()
            assert (err <= tol).all(), (b, t, (err / tol.clamp_min(1e-30)).max())
            z = (Q[b, t, 0].double() @ K[b, base].double().T) * (scale * math.log2(math.e))
            tops = torch.stack([c.max() for c in z.split(TILE)])
            moved += int((tops[2:] > tops[:-2] + 8).sum())  # one stream's next tile
    assert moved > 0


# --------------------------------------------------------------------- scores
def integer_inputs(B, T, H, S, g):
    q = torch.randint(-3, 4, (B, T, H, 128), generator=g).bfloat16()
    w = torch.tensor([-1.0, -0.5, 0.5, 1.0])[torch.randint(0, 4, (B, T, H), generator=g)].bfloat16()
    k8 = torch.randint(-4, 5, (B, S, 128), generator=g, dtype=torch.int8).float().to(torch.float8_e4m3fn)
    scale = torch.tensor([0.25, 1.0, 2.0])[torch.randint(0, 3, (B, S), generator=g)]
    return q, w, k8.view(torch.uint8), scale


SCORE_CASES = [
    # B, T, H_I, S_max, ragged drafts, at least: tiles of the longest part, parts of a CTA
    (300, 3, 64, 300, False, 1, 2),   # one accumulator, several parts
    (200, 9, 64, 300, True, 1, 2),    # two accumulators and one, part by part
    (150, 17, 32, 700, True, 1, 2),
    (2, 16, 64, 60000, False, 7, 1),  # the rings of the 512-column form go round
    (2, 4, 64, 120000, False, 7, 1),  # .. of the 256-column form
    (3, 13, 32, 50001, True, 4, 1),
    (61, 10, 64, 4001, True, 9, 2),   # long parts, and a change of part
    (31, 16, 64, 7001, False, 9, 2),
]


@pytest.mark.parametrize("B,T,H,S,ragged,tiles,parts", SCORE_CASES)
def test_scores_over_many_tiles_and_parts(ic, ctx, B, T, H, S, ragged, tiles, parts):
    """Integer inputs, every partial sum exact: every score of every row is equal."""
    g = torch.Generator().manual_seed(S + B)
    q, w, k8, scale = integer_inputs(B, T, H, S, g)
    draft = [1 + (5 * b) % T if ragged else T for b in range(B)]
    prefix = [S - T - (37 * b) % 130 for b in range(B)]
    group = (256 if T * H <= 256 else 512) // H
    split = parts_of(units_of(prefix, draft, 1, group), 1)
    assert max(max(p) for p in split) >= tiles and max(len(p) for p in split) >= parts
    mask = chains(B, T)
    ld = (S + 3) // 4 * 4 + 4
    out = torch.full((B * T, ld), 777.0, device="cuda")
    ic.ic_index_score_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(),
                           torch.tensor(prefix, dtype=torch.int32).cuda(), out,
                           draft_len=torch.tensor(draft, dtype=torch.int32).cuda(), tree_mask=mask.cuda())
    ctx.sync_status()
    got = out.view(B, T, ld)
    for b in range(B):
        n, m = prefix[b], draft[b]
        end = n + m
        k = k8[b, :end].cuda().view(torch.float8_e4m3fn).double()
        hidden = ~ref.visible(n, m, mask[b], m).cuda()
        for t in range(m) if end < 2000 else {0, m // 2, m - 1}:
            dots = (q[b, t].cuda().double() @ k.T).clamp_min(0)
            want = (w[b, t].cuda().double() @ dots) * scale[b, :end].cuda().double()
            want[n:][hidden[t]] = -math.inf
            assert torch.equal(got[b, t, :end].double(), want), (b, t)
        assert (got[b, :m, end:] == 777.0).all() and (got[b, m:] == 777.0).all()


# ------------------------------------------------------- infinities in queries
@pytest.mark.parametrize("T,H", [(3, 64), (3, 32), (12, 64)])
def test_scores_of_infinite_queries(ic, ctx, T, H):
    """ReLU of -inf is 0 and of +inf is +inf; inf * 0 and inf - inf are NaN, as in the formula."""
    B, S = 2, 300
    g = torch.Generator().manual_seed(T * H)
    q, w, k8, scale = integer_inputs(B, T, H, S, g)
    inf = math.inf
    q[0, 0, 5, 7] = -inf
    q[0, 1, 3, 0], q[0, 1, 9, 1], w[0, 1, 9] = inf, -inf, 0.0
    q[1, 2, H - 1, 64:66] = torch.tensor([inf, -inf]).bfloat16()
    q[1, 1, :, 0] = -inf
    prefix = [290, 100]
    out = torch.zeros((B * T, S), device="cuda")
    ic.ic_index_score_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(),
                           torch.tensor(prefix, dtype=torch.int32).cuda().sub_(T - 10 if T > 10 else 0), out)
    ctx.sync_status()
    if T > 10:
        prefix = [p - (T - 10) for p in prefix]
    got = out.cpu().double().view(B, T, S)
    odd = 0
    for b in range(B):
        end = prefix[b] + T
        k = k8[b, :end].view(torch.float8_e4m3fn).double()
        dots = torch.stack([(q[b, t].double()[:, None, :] * k[None]).sum(-1) for t in range(T)])
        want = (w[b].double()[:, :, None] * torch.relu(dots)).sum(1) * scale[b, :end].double()
        see = ref.visible(prefix[b], T, None, T)
        want[:, prefix[b]:][~see] = -inf
        odd += int((dots == -inf).sum())
        x = got[b, :, :end]
        assert torch.equal(torch.isnan(x), torch.isnan(want))
        fin = ~torch.isnan(want)
        assert torch.equal(x[fin], want[fin])
    assert odd > 100


def test_scores_of_infinite_queries_with_large_weights(ic, ctx):
    """A head whose query holds an infinity keeps its weight as it is: 0 times a large one is 0."""
    B, T, H, S = 1, 2, 32, 200
    g = torch.Generator().manual_seed(9)
    q, w, k8, scale = integer_inputs(B, T, H, S, g)
    k8[0, :, 3] = torch.ones(()).to(torch.float8_e4m3fn).view(torch.uint8)  # 1 at 3
    q[0, 0, 4, :], q[0, 0, 4, 3] = 0, -math.inf
    w[0, 0, 4] = 2.0 ** 100
    k = k8[0].view(torch.float8_e4m3fn).double()
    out = torch.zeros((B * T, S), device="cuda")
    ic.ic_index_score_tree(ctx, q.cuda(), w.cuda(), k8.cuda(), scale.cuda(),
                           torch.tensor([190], dtype=torch.int32).cuda(), out)
    ctx.sync_status()
    rest = [j for j in range(H) if j != 4]
    want = (w[0, 0, rest].double()[:, None] * (q[0, 0, rest].double() @ k[:190].T).clamp_min(0)).sum(0)
    assert torch.equal(out[0, :190].cpu().double(), want * scale[0, :190].double())
