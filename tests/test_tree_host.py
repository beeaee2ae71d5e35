"""Drafted-token operators and norm + rotation without a GPU: what the C
entry points and the binding refuse before anything is launched, and checks
of the 64-bit forms in tree_ref.py (against loops written out, and against
mistakes planted in them)."""
import ctypes
import math
import types

import pytest
import torch

from tests import tree_ref


@pytest.fixture(scope="module")
def ic():
    from cross_layer_top_b200 import build
    build.build()
    from cross_layer_top_b200 import indexcache
    return indexcache


# A context that the binding's own checks get to see: CPU tensors report
# device -1, so they pass for tensors of the context's device and every check
# behind that one can fail in its turn.  Nothing here may reach the library.
@pytest.fixture()
def ctx(ic, monkeypatch):
    def reached(*a):
        raise AssertionError("the binding let a bad call through")
    for name in ("ic_qk_norm_rope", "ic_index_score_tree", "ic_index_fp_tree", "ic_tree_attn"):
        monkeypatch.setattr(ic._lib, name, reached)
    monkeypatch.setattr(ic, "_ctx_stream", lambda ctx, stream: 0)
    return types.SimpleNamespace(handle=None, device=-1)


# ------------------------------------------------------------- C entry points
def test_null_context(ic):
    z, n = 0, None
    head = ic.ic_head_io()
    assert ic._lib.ic_qk_norm_rope(n, ctypes.byref(head), 1, 1, z, 1, z) == ic.IC_ERR_INVALID_ARG
    assert ic._lib.ic_index_score_tree(n, z, z, z, z, z, z, z, 1, 1, 1, 32, 128, z, 4,
                                       z) == ic.IC_ERR_INVALID_ARG
    assert ic._lib.ic_index_fp_tree(n, z, z, z, z, z, z, z, 1, 1, 1, 32, 128, 1, z,
                                    z) == ic.IC_ERR_INVALID_ARG
    assert ic._lib.ic_tree_attn(n, z, z, z, z, z, z, z, 1, 1, 1, 64, 0, 64, 1, 0.0, z,
                                z) == ic.IC_ERR_INVALID_ARG


def test_descriptor_layout(ic):
    """The packed form of the descriptors is the structure's own layout."""
    import struct
    assert struct.calcsize(ic._HEAD_IO) == ctypes.sizeof(ic.ic_head_io)
    names = [f[0] for f in ic.ic_head_io._fields_]
    vals = [float(i) if n == "eps" else i + 1 for i, n in enumerate(names)]
    io = ic.ic_head_io()
    struct.pack_into(ic._HEAD_IO, io, 0, *vals)
    for n, v in zip(names, vals):
        assert getattr(io, n) == v, n


def some_heads(rows, strided, fp8):
    g = torch.Generator().manual_seed(rows)
    width = 4 * 64 + 64 + 128
    fused = torch.randn((rows, width + (8 if strided else 0)), generator=g).bfloat16()
    q, k = fused[:, :256].unflatten(1, (4, 64)), fused[:, 256:320].unflatten(1, (1, 64))
    i = fused[:, 320:448].unflatten(1, (1, 128))
    rope, rope_i = torch.zeros((50, 64)), torch.zeros((50, 32))
    slot = torch.arange(rows)
    heads = [dict(x=q, norm="rms", weight=torch.ones(64), rope=rope, out=torch.zeros(rows, 4, 64).bfloat16()),
             dict(x=k, norm="rms", weight=torch.ones(64), eps=1e-5, rope=rope, slot=slot,
                  out=torch.zeros(rows + 9, 64).bfloat16()),
             dict(x=k, slot=slot, out=torch.zeros(rows + 3, 1, 64).bfloat16(), weight=None, bias=None)]
    if fp8:
        heads.append(dict(x=i, norm="layer", weight=torch.ones(128), bias=torch.zeros(128), rope=rope_i,
                          interleaved=True, slot=slot, out8=torch.zeros((rows, 1, 128), dtype=torch.uint8),
                          out_scale=torch.zeros(rows, 1)))
    return heads


@pytest.mark.parametrize("rows", [0, 1, 7])
@pytest.mark.parametrize("strided", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_both_ways_to_descriptors_agree(ic, ctx, rows, strided, fp8):
    heads = some_heads(rows, strided, fp8)
    slow, n, n_pos = ic.make_head_ios(ctx, heads)
    packed = ic._tensors.pack(heads, ctx.device)
    assert packed is not None and packed[1:] == (n, n_pos) == (rows, 50)
    size = ctypes.sizeof(ic.ic_head_io)
    assert len(packed[0]) == size * len(heads)
    for i in range(len(heads)):
        fast = ic.ic_head_io.from_buffer_copy(packed[0], i * size)
        for name, _ in ic.ic_head_io._fields_:
            assert getattr(fast, name) == getattr(slow[i], name), (i, name)


def test_fast_descriptors_leave_the_rest(ic, ctx):
    ok = some_heads(3, False, True)
    assert ic._tensors.pack(ok, -1) is not None
    assert ic._tensors.pack(ok, 0) is None and ic._tensors.pack(tuple(ok), -1) is None
    assert ic._tensors.pack([], -1) is None and ic._tensors.pack(ok[:1] * 9, -1) is None
    x = ok[0]["x"]
    for bad in (dict(x=None), dict(x=3), dict(x=x.float()), dict(x=x[0]), dict(x=x.transpose(1, 2)),
                dict(norm="l2"), dict(norm=1), dict(eps=1), dict(eps=None), dict(weight=torch.ones(63)),
                dict(weight=torch.ones(64).double()), dict(bias=[0.0]), dict(rope=torch.zeros(50)),
                dict(rope=torch.zeros((49, 64))), dict(interleaved=1), dict(out=None), dict(rows=3),
                dict(out8=torch.zeros((3, 4, 64), dtype=torch.uint8)), dict(slot=torch.arange(2)),
                dict(slot=torch.arange(3).int()), dict(out=torch.zeros((4, 4, 64)).bfloat16()),
                dict(x=x.to("meta"))):
        assert ic._tensors.pack([ok[1], dict(ok[0], **bad)], -1) is None, bad
    with pytest.raises(TypeError):
        ic._tensors.pack(ok)
    with pytest.raises(TypeError):
        ic._tensors.pack(ok, "cuda")


def test_fast_argument_checks(ic):
    t = torch.zeros((2, 3, 8), dtype=torch.bfloat16)
    ptr, cache = ic._tensors.ptr, ic._tensors.cache
    assert ptr(t, torch.bfloat16, -1, None) == t.data_ptr() == ptr(t, torch.bfloat16, -1, (2, 3, 8))
    assert ptr(t, torch.bfloat16, -1, t.shape) == t.data_ptr()
    assert ptr(t[1], torch.bfloat16, -1, (3, 8)) == t.data_ptr() + 48
    assert ptr(t[:0], torch.bfloat16, -1, (0, 3, 8)) is not None
    for bad in ((t, torch.float16, -1, None), (t, torch.bfloat16, 0, None), (t, torch.bfloat16, -1, (2, 3)),
                (t, torch.bfloat16, -1, (2, 3, 9)), (t, torch.bfloat16, -1, [2, 3, 8]),
                (t, torch.bfloat16, -1, (2, 3, 8.5)), (t[..., :4], torch.bfloat16, -1, None),
                (t.to("meta"), torch.bfloat16, -1, None), (3, torch.bfloat16, -1, None), (t, "bf16", -1, None),
                (t.to_sparse(), torch.bfloat16, -1, None)):
        assert ptr(*bad) is None, bad
    kv = torch.zeros((2, 2, 5, 8), dtype=torch.bfloat16)
    assert cache(kv[:, 1], -1, 2, 5, 8) == (kv.data_ptr() + 80, 80)
    assert cache(kv[:1, 1], -1, 1, 5, 8) == (kv.data_ptr() + 80, 40)
    assert cache(t[:, :1], -1, 2, 1, 8) == (t.data_ptr(), 24)
    for bad in ((kv[:, 1].float(), -1, 2, 5, 8), (kv[:, 1], 0, 2, 5, 8), (kv[:, 1], -1, 2, 4, 8),
                (kv[:, 1], -1, 3, 5, 8), (kv[:, 1], -1, 2, 5, 4), (kv, -1, 2, 5, 8), (kv[0, ..., :4], -1, 2, 5, 4),
                (kv[0].transpose(1, 2), -1, 2, 8, 5), (None, -1, 2, 5, 8)):
        assert cache(*bad) is None, bad
    for call in (lambda: ptr(t), lambda: ptr(t, torch.bfloat16, "cuda", None), lambda: cache(kv, -1, 2, 5)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ binding
def score_args(B=2, T=3, H=32, S=100, d=128):
    return [torch.zeros((B, T, H, d), dtype=torch.bfloat16), torch.zeros((B, T, H), dtype=torch.bfloat16),
            torch.zeros((B, S, d), dtype=torch.uint8), torch.zeros((B, S)),
            torch.zeros(B, dtype=torch.int32)]


@pytest.mark.parametrize("at,bad", [
    (0, torch.zeros((2, 3, 32, 128))), (1, torch.zeros((2, 3, 31), dtype=torch.bfloat16)),
    (2, torch.zeros((2, 100, 128))), (2, torch.zeros((2, 100, 64), dtype=torch.uint8)),
    (2, torch.zeros((2, 128, 100), dtype=torch.uint8).transpose(1, 2)), (3, torch.zeros((2, 99))),
    (4, torch.zeros(2, dtype=torch.int64)), (4, torch.zeros(3, dtype=torch.int32))])
def test_score_refusals(ic, ctx, at, bad):
    args = score_args()
    args[at] = bad
    scores, idx = torch.zeros((6, 100)), torch.zeros((6, 8), dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        ic.ic_index_score_tree(ctx, *args, scores)
    with pytest.raises((TypeError, ValueError)):
        ic.ic_index_fp_tree(ctx, *args, 8, idx)


def test_score_output_and_option_refusals(ic, ctx):
    args = score_args()
    idx = torch.zeros((6, 8), dtype=torch.int32)
    for scores in (torch.zeros((5, 100)), torch.zeros(600), torch.zeros((6, 100), dtype=torch.float64),
                   torch.zeros((6, 200))[:, :100]):
        with pytest.raises((TypeError, ValueError)):
            ic.ic_index_score_tree(ctx, *args, scores)
    for bad in (idx[:5], idx.long(), torch.zeros((6, 9), dtype=torch.int32)):
        with pytest.raises((TypeError, ValueError)):
            ic.ic_index_fp_tree(ctx, *args, 8, bad)
    for opt in (dict(draft_len=torch.zeros(3, dtype=torch.int32)), dict(draft_len=torch.zeros(2)),
                dict(tree_mask=torch.zeros((2, 3), dtype=torch.int32)),
                dict(tree_mask=torch.zeros((2, 4), dtype=torch.int64))):
        with pytest.raises((TypeError, ValueError)):
            ic.ic_index_score_tree(ctx, *args, torch.zeros((6, 100)), **opt)
        with pytest.raises((TypeError, ValueError)):
            ic.ic_index_fp_tree(ctx, *args, 8, idx, **opt)
    far = types.SimpleNamespace(handle=None, device=0)
    with pytest.raises(ValueError, match="cuda:0"):
        ic.ic_index_score_tree(far, *args, torch.zeros((6, 100)))


def test_attention_refusals(ic, ctx):
    B, T, Hq, d, S = 2, 3, 4, 64, 100
    Q = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16)
    kv = torch.zeros((B, 2, S, d), dtype=torch.bfloat16)
    K, V = kv[:, 0], kv[:, 1]
    p, out = torch.zeros(B, dtype=torch.int32), torch.zeros_like(Q)
    wide = torch.zeros((B, S, 2 * d), dtype=torch.bfloat16)
    bad = [
        (Q.float(), K, V, p, out, {}), (Q, K.float(), V, p, out, {}), (Q, K, V[:, :99], p, out, {}),
        (Q, wide[..., :d], wide[..., d:], p, out, {}), (Q, K, V.contiguous(), p, out, {}),
        (Q, K[:1], V[:1], p, out, {}), (Q, K, V, p.long(), out, {}), (Q, K, V, p, out[:, :2], {}),
        (Q, K, V, p, out.float(), {}), (Q.transpose(1, 2), K, V, p, out, {}),
        (Q, K, V, p, out, dict(idx=torch.zeros((3, 8), dtype=torch.int32))),
        (Q, K, V, p, out, dict(idx=torch.zeros((2, 8), dtype=torch.int64))),
        (Q, K, V, p, out, dict(idx=torch.zeros((2, 0), dtype=torch.int32))),
        (Q, K, V, p, out, dict(draft_len=torch.zeros((2, 1), dtype=torch.int32))),
        (Q, K, V, p, out, dict(tree_mask=torch.zeros((2, 3)))),
    ]
    for q, k, v, pre, o, opt in bad:
        with pytest.raises((TypeError, ValueError)):
            ic.ic_tree_attn(ctx, q, k, v, pre, o, **opt)


def test_head_refusals(ic, ctx):
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    o, pos = torch.zeros_like(x), torch.zeros(4, dtype=torch.int32)
    o8, sc = torch.zeros((4, 2, 64), dtype=torch.uint8), torch.zeros((4, 2))
    rope = torch.zeros((10, 64))
    bad = [
        dict(x=x.float(), out=o), dict(x=x[0], out=o), dict(x=x), dict(x=x, out=o, out8=o8),
        dict(x=x, out=o[:3]), dict(x=x, out=o.float()), dict(x=x, out8=o, out_scale=sc),
        dict(x=x, out8=o8, out_scale=sc[:3]), dict(x=x, out=o, wieght=torch.zeros(64)),
        dict(x=x, out=o, norm="rms", weight=torch.zeros(32)),
        dict(x=x, out=o, norm="rms", weight=torch.zeros(64, dtype=torch.bfloat16)),
        dict(x=x, out=o, rope=rope.double()), dict(x=x, out=o, rope=rope.t().contiguous().t()),
        dict(x=x, out=o, slot=torch.zeros(4, dtype=torch.int32)),
        dict(x=x, out=o, slot=torch.zeros(3, dtype=torch.int64)), dict(x=x.transpose(1, 2), out=o),
    ]
    for hd in bad:
        with pytest.raises((TypeError, ValueError)):
            ic.ic_qk_norm_rope(ctx, [hd], pos)
    ok = dict(x=x, out=o, rope=rope)
    for heads in ([ok, dict(x=x[:3], out=o[:3])], [ok, dict(x=x, out=o, rope=rope[:9])]):
        with pytest.raises(ValueError):
            ic.ic_qk_norm_rope(ctx, heads, pos)
    for p in (pos.long(), pos[:3]):
        with pytest.raises((TypeError, ValueError)):
            ic.ic_qk_norm_rope(ctx, [ok], p)


# ---------------------------------------------------------- the 64-bit forms
def loops_score(q, w, k8, scale, prefix, draft, mask):
    k = k8.view(torch.float8_e4m3fn).double()
    out = torch.full((draft, prefix + draft), -math.inf, dtype=torch.float64)
    for t in range(draft):
        for s in range(prefix + draft):
            u = s - prefix
            if u >= 0 and not (u <= t if mask is None else int(mask[t]) >> u & 1):
                continue
            out[t, s] = float(scale[s]) * sum(
                float(w[t, j]) * max(float((q[t, j].double() * k[s]).sum()), 0.0)
                for j in range(q.shape[1]))
    return out


def loops_attn(Q, K, V, prefix, draft, mask, idx, scale):
    out = torch.zeros((draft,) + tuple(Q.shape[1:]), dtype=torch.float64)
    base = list(range(prefix)) if idx is None else [int(i) for i in idx if i >= 0]
    for t in range(draft):
        seen = base + [prefix + u for u in range(draft)
                       if (u <= t if mask is None else int(mask[t]) >> u & 1)]
        for h in range(Q.shape[1]):
            if seen:
                z = torch.stack([(Q[t, h].double() * K[s].double()).sum() * scale for s in seen])
                p = torch.exp(z - z.max())
                out[t, h] = sum(pi / p.sum() * V[s].double() for pi, s in zip(p, seen))
    return out


def score_case():
    g = torch.Generator().manual_seed(5)
    return (torch.randn((4, 3, 8), generator=g).bfloat16(), torch.randn((4, 3), generator=g).bfloat16(),
            torch.randn((9, 8), generator=g).to(torch.float8_e4m3fn).view(torch.uint8),
            torch.rand(9, generator=g) + 0.5)


def attn_case():
    g = torch.Generator().manual_seed(6)
    return [torch.randn(s, generator=g).bfloat16() for s in ((4, 2, 16), (9, 16), (9, 16))]


TREE = torch.tensor([0b1, 0b11, 0b101, 0])


@pytest.mark.parametrize("mask", [None, TREE])
@pytest.mark.parametrize("prefix,draft", [(5, 4), (0, 4), (6, 1), (5, 0)])
def test_scores_form(prefix, draft, mask):
    a = score_case()
    got, tol = tree_ref.tree_scores(*a, prefix, draft, mask)
    want = loops_score(*a, prefix, draft, mask)
    assert torch.equal(got == -math.inf, want == -math.inf)
    fin = want != -math.inf
    assert ((got - want)[fin].abs() <= 1e-12).all() and (tol[fin] < 1e-3).all()


@pytest.mark.parametrize("idx", [None, torch.tensor([4, -1, 0, 4])])
@pytest.mark.parametrize("mask", [None, TREE])
@pytest.mark.parametrize("prefix,draft", [(5, 4), (5, 1), (5, 0)])
def test_attention_form(prefix, draft, mask, idx):
    a = attn_case()
    got, tol = tree_ref.tree_attn(*a, prefix, draft, mask, idx, 0.25)
    want = loops_attn(*a, prefix, draft, mask, idx, 0.25)
    assert ((got - want).abs() <= 1e-12).all()
    assert (tol < 0.05).all()


def test_a_row_that_sees_nothing_is_zero():
    a = attn_case()
    got, _ = tree_ref.tree_attn(*a, 0, 4, TREE, None, 0.25)
    assert (got[3] == 0).all() and (got[0] != 0).any()


@pytest.mark.parametrize("norm", [None, "rms", "layer"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_form(norm, interleaved):
    g = torch.Generator().manual_seed(7)
    x = torch.randn((3, 2, 32), generator=g).bfloat16()
    weight = torch.rand(32, generator=g) + 0.5 if norm else None
    bias = torch.randn(32, generator=g) if norm == "layer" else None
    ang = torch.rand((6, 8), generator=g) * 6
    rope = torch.cat([torch.cos(ang), torch.sin(ang)], 1)
    pos = torch.tensor([5, 0, 2])
    got, tol = tree_ref.norm_rope(x, norm, weight, bias, 1e-5, rope, pos, interleaved)
    for r in range(3):
        for h in range(2):
            y = [float(v) for v in x[r, h]]
            if norm:
                mu = sum(y) / 32 if norm == "layer" else 0.0
                y = [v - mu for v in y]
                rms = math.sqrt(sum(v * v for v in y) / 32 + 1e-5)
                y = [v / rms * float(weight[i]) + (float(bias[i]) if norm == "layer" else 0.0)
                     for i, v in enumerate(y)]
            z = list(y)
            for i in range(8):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
                c, s = float(rope[pos[r], i]), float(rope[pos[r], 8 + i])
                z[a], z[b] = y[a] * c - y[b] * s, y[b] * c + y[a] * s
            assert ((got[r, h] - torch.tensor(z, dtype=torch.float64)).abs() <= 1e-12).all()
    assert (tol < 1e-3).all()


# Mistakes that a kernel could make, made in the plain forms: the bounds the
# GPU tests use tell them apart.
def test_bounds_reject_a_wrong_score():
    q, w, k8, scale = score_case()
    want, tol = tree_ref.tree_scores(q, w, k8, scale, 5, 4, TREE)
    fin = want != -math.inf
    no_relu = torch.einsum("th,thd,sd->ts", w.double(), q.double(),
                           k8.view(torch.float8_e4m3fn).double()) * scale.double()
    dropped, _ = tree_ref.tree_scores(q[:, :2], w[:, :2], k8, scale, 5, 4, TREE)
    shifted, _ = tree_ref.tree_scores(q, w, k8, scale.roll(1), 5, 4, TREE)
    for wrong in (no_relu, dropped, shifted):
        assert not ((wrong - want)[fin].abs() <= tol[fin]).all()
    chain, _ = tree_ref.tree_scores(q, w, k8, scale, 5, 4, None)
    assert not torch.equal(chain == -math.inf, want == -math.inf)


def test_bounds_reject_a_wrong_attention():
    Q, K, V = attn_case()
    want, tol = tree_ref.tree_attn(Q, K, V, 5, 4, TREE, None, 0.25)
    for wrong, _ in (tree_ref.tree_attn(Q, K, V, 5, 4, None, None, 0.25),
                     tree_ref.tree_attn(Q, K, V, 5, 4, TREE, torch.arange(1, 5), 0.25),
                     tree_ref.tree_attn(Q, K, V, 5, 4, TREE, torch.tensor([0, 1, 2, 3, 4, 4]), 0.25),
                     tree_ref.tree_attn(Q, K, V, 5, 4, TREE, None, 0.27),
                     tree_ref.tree_attn(Q, K, V.roll(1, 0), 5, 4, TREE, None, 0.25)):
        assert not ((wrong - want).abs() <= tol).all()


def test_bounds_reject_a_wrong_rotation():
    g = torch.Generator().manual_seed(8)
    x = torch.randn((3, 2, 32), generator=g).bfloat16()
    ang = torch.rand((6, 16), generator=g) * 6
    rope = torch.cat([torch.cos(ang), torch.sin(ang)], 1)
    pos = torch.tensor([5, 1, 2])
    want, tol = tree_ref.norm_rope(x, "rms", None, None, 1e-5, rope, pos, False)
    tol = tol + want.abs() * tree_ref.UBF16  # the store
    back = torch.cat([torch.cos(ang), -torch.sin(ang)], 1)
    for wrong, _ in (tree_ref.norm_rope(x, "rms", None, None, 1e-5, rope, pos, True),
                     tree_ref.norm_rope(x, "rms", None, None, 1e-5, back, pos, False),
                     tree_ref.norm_rope(x, "rms", None, None, 1e-5, rope, pos - 1, False),
                     tree_ref.norm_rope(x, "layer", None, None, 1e-5, rope, pos, False)):
        assert not ((wrong - want).abs() <= tol).all()
