"""ic_qk_norm_rope against its 64-bit form: norms, rotations, head layouts,
output types, slots, strides, refusals.  Bounds from tests/tree_ref.py."""
import numpy as np
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


def table(n_pos, dr):
    f = 10000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64) / dr)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def check_bf16(got, z, tol):
    got = got.double()
    bad = (got - z).abs() > tol + (z.abs() + tol) * ref.UBF16
    assert not bad.any(), (got - z).abs().max()


def check_fp8(got8, scale, z, tol):
    """got8 uint8 [.., d], scale [..]: the scale within its roundings, the values within half a step."""
    top = z.abs().amax(-1).clamp_min(1e-12)
    s = scale.double()
    assert ((s - top / 448).abs() <= tol.amax(-1) / 448 + top / 448 * 4 * ref.U32).all()
    v = got8.view(torch.float8_e4m3fn).double() * s[..., None]
    half = torch.maximum(z.abs() * ref.UE4M3, s[..., None] * 2.0 ** -10)
    assert ((v - z).abs() <= half * (1 + 1e-5) + tol * 1.1).all()


CASES = [
    # rows, H, d, d_rot, norm, bias, interleaved, fp8, strided
    (1, 1, 128, 128, "rms", False, False, False, False),
    (1, 1, 32, 16, "layer", True, True, True, False),
    (7, 16, 128, 128, "rms", False, False, False, True),
    (33, 16, 128, 64, "rms", False, True, False, True),
    (5, 64, 128, 64, None, False, False, False, True),
    (65, 64, 128, 64, None, False, False, True, True),
    (129, 1, 128, 64, "layer", True, False, True, True),
    (31, 3, 64, 64, "rms", False, False, False, True),
    (30, 7, 64, 48, "layer", False, False, False, True),
    (513, 4, 32, 32, "rms", False, True, True, True),
    (19, 5, 32, 16, "layer", True, False, False, False),
    (100, 1, 128, 0, None, False, False, False, True),
    (257, 2, 64, 0, "rms", False, False, True, False),
    (9, 130, 128, 112, "layer", True, False, False, False),
]


@pytest.mark.parametrize("rows,H,d,dr,norm,bias,inter,fp8,strided", CASES)
def test_one_tensor(ic, ctx, rows, H, d, dr, norm, bias, inter, fp8, strided):
    g = torch.Generator().manual_seed(rows * 131 + H)
    width = H * d + (24 if strided else 0)
    base = (torch.randn((rows, width), generator=g) * 2 + 0.3).bfloat16()
    off = 8 if strided else 0
    x = base[:, off:off + H * d].unflatten(1, (H, d))
    xg = base.cuda()[:, off:off + H * d].unflatten(1, (H, d))
    wt = 1 + 0.2 * torch.randn(d, generator=g) if norm else None
    bs = 0.2 * torch.randn(d, generator=g) if bias else None
    rope = table(5000, dr) if dr else None
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32)
    pos[0] = 4999
    z, tol = ref.norm_rope(x, norm, wt, bs, 1e-6, rope, pos, inter)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    head = dict(x=xg, norm=norm, weight=cu(wt), bias=cu(bs), eps=1e-6, rope=cu(rope),
                interleaved=inter)
    if fp8:
        o8 = torch.full((rows, H, d), 0x55, dtype=torch.uint8, device="cuda")
        sc = torch.full((rows, H), -1.0, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out8=o8, out_scale=sc)], pos.cuda())
        ctx.sync_status()
        check_fp8(o8.cpu(), sc.cpu(), z, tol)
    else:
        o = torch.full((rows, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out=o)], pos.cuda())
        ctx.sync_status()
        check_bf16(o.cpu(), z, tol)
        if norm is None and rope is None:
            assert torch.equal(o.cpu(), x)


def test_slots_scatter_and_leave_the_rest(ic, ctx):
    """Cache writes: distinct slots in any order, -1 writes nothing, other rows keep their bytes."""
    rows, cache = 77, 300
    g = torch.Generator().manual_seed(3)
    x = torch.randn((rows, 1, 128), generator=g).bfloat16()
    slot = torch.randperm(cache, generator=g)[:rows]
    slot[::9] = -1
    K = torch.full((cache, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    k8 = torch.full((cache, 128), 0x11, dtype=torch.uint8, device="cuda")
    sc = torch.full((cache,), 5.0, device="cuda")
    s = slot.cuda()
    ic.ic_qk_norm_rope(ctx, [dict(x=x.cuda(), out=K, slot=s),
                             dict(x=x.cuda(), out8=k8, out_scale=sc, slot=s)])
    ctx.sync_status()
    live = slot >= 0
    want = torch.full((cache, 128), 7.0, dtype=torch.bfloat16)
    want[slot[live]] = x[live, 0]
    assert torch.equal(K.cpu(), want)
    rest = torch.ones(cache, dtype=torch.bool)
    rest[slot[live]] = False
    assert (k8.cpu()[rest] == 0x11).all() and (sc.cpu()[rest] == 5.0).all()
    check_fp8(k8.cpu()[slot[live]], sc.cpu()[slot[live]], x[live, 0].double(),
              torch.zeros(int(live.sum()), 128, dtype=torch.float64))


def test_two_tensors_share_a_cache(ic, ctx):
    """K and V as halves of one [B, 2, S, d] cache: the slots say which rows are whose."""
    B, S, d, rows = 3, 50, 128, 37
    g = torch.Generator().manual_seed(12)
    k, v = (torch.randn((rows, 1, d), generator=g).bfloat16() for _ in range(2))
    at = torch.randperm(B * S, generator=g)[:rows]
    b, s = at // S, at % S
    kv = torch.full((B, 2, S, d), 7.0, dtype=torch.bfloat16, device="cuda")
    rope = table(S, d)
    flat = kv.view(B * 2 * S, 1, d)
    pos = s.int()
    ic.ic_qk_norm_rope(ctx, [
        dict(x=k.cuda(), norm="rms", rope=rope.cuda(), out=flat, slot=(b * 2 * S + s).cuda()),
        dict(x=v.cuda(), out=flat, slot=((b * 2 + 1) * S + s).cuda())], pos.cuda())
    ctx.sync_status()
    got = kv.cpu()
    z, tol = ref.norm_rope(k, "rms", None, None, 1e-6, rope, pos, False)
    check_bf16(got[b, 0, s], z[:, 0], tol[:, 0])
    assert torch.equal(got[b, 1, s], v[:, 0])
    rest = torch.ones((B, S), dtype=torch.bool)
    rest[b, s] = False
    assert (got[:, 0][rest] == 7).all() and (got[:, 1][rest] == 7).all()


def test_zero_and_extreme_rows(ic, ctx):
    """A zero vector keeps a positive scale; rows of the largest and least magnitudes stay finite."""
    x = torch.zeros((4, 1, 128), dtype=torch.bfloat16)
    x[1] = 3e38
    x[1, 0, ::2] = -3e38
    x[2] = 1e-38
    x[3, 0, 5] = 1.0
    o8 = torch.zeros((4, 1, 128), dtype=torch.uint8, device="cuda")
    sc = torch.zeros((4, 1), device="cuda")
    o = torch.zeros((4, 1, 128), dtype=torch.bfloat16, device="cuda")
    ic.ic_qk_norm_rope(ctx, [dict(x=x.cuda(), out8=o8, out_scale=sc), dict(x=x.cuda(), out=o)])
    ctx.sync_status()
    assert torch.equal(o.cpu(), x)
    assert (sc > 0).all() and torch.isfinite(sc).all()
    v = o8.cpu().view(torch.float8_e4m3fn).double()
    assert (v[0] == 0).all() and (v[2] == 0).all()
    assert (v[1].abs() == 448).all()
    assert v[3, 0, 5] == 448 and v[3].abs().sum() == 448


def test_not_a_number_stays_in_its_vector(ic, ctx):
    x = torch.ones((3, 4, 128), dtype=torch.bfloat16)
    x[1, 2, 77] = float("nan")
    o = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device="cuda")
    ic.ic_qk_norm_rope(ctx, [dict(x=x.cuda(), norm="rms", out=o)])
    ctx.sync_status()
    nan = torch.isnan(o.cpu())
    assert nan[1, 2].all() and nan.sum() == 128


def test_many_tensors_equal_one_by_one(ic, ctx):
    """Eight tensors of mixed shapes in one launch give the bytes of eight launches."""
    rows = 37
    g = torch.Generator().manual_seed(9)
    rope = {d: table(700, d).cuda() for d in (16, 32, 64, 128)}
    pos = torch.randint(0, 700, (rows,), generator=g, dtype=torch.int32).cuda()
    heads = []
    for i, (H, d, dr, norm) in enumerate([(16, 128, 128, "rms"), (1, 128, 64, "layer"), (1, 64, 0, None),
                                          (64, 128, 64, None), (3, 32, 16, "rms"), (4, 64, 32, None),
                                          (7, 32, 32, "layer"), (2, 128, 128, "rms")]):
        x = torch.randn((rows, H, d), generator=g).bfloat16().cuda()
        hd = dict(x=x, norm=norm, rope=rope.get(dr), interleaved=bool(i & 1))
        if i % 3 == 1:
            hd |= dict(out8=torch.zeros((rows, H, d), dtype=torch.uint8, device="cuda"),
                       out_scale=torch.zeros((rows, H), device="cuda"))
        else:
            hd |= dict(out=torch.zeros((rows, H, d), dtype=torch.bfloat16, device="cuda"))
        heads.append(hd)
    ic.ic_qk_norm_rope(ctx, heads, pos)
    for hd in heads:
        one = {k: (torch.zeros_like(v) if k in ("out", "out8", "out_scale") else v)
               for k, v in hd.items()}
        ic.ic_qk_norm_rope(ctx, [one], pos)
        for k in ("out", "out8", "out_scale"):
            if k in hd:
                assert torch.equal(hd[k], one[k])
    ctx.sync_status()


def test_bad_positions_and_slots_are_reported(ic, ctx):
    rows = 20
    x = torch.ones((rows, 2, 64), dtype=torch.bfloat16, device="cuda")
    rope = table(50, 64).cuda()
    for bad in (-1, 50, 2 ** 31 - 1):
        pos = torch.full((rows,), 3, dtype=torch.int32)
        pos[7] = bad
        o = torch.full((rows, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(x=x, rope=rope, out=o)], pos.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE and "position" in str(e.value)
        kept = (o == 9.0).flatten(1).all(1).cpu()
        assert kept[7] and kept.sum() == 1
    for bad in (-2, 40, 2 ** 62):
        slot = torch.arange(rows, dtype=torch.int64)
        slot[11] = bad
        o = torch.full((40, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(x=x, out=o, slot=slot.cuda())])
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE and "slot" in str(e.value)
        kept = (o == 9.0).flatten(1).all(1).cpu()
        assert kept[11] and kept.sum() == 21
    ctx.sync_status()


def test_refusals(ic, ctx):
    x = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    o = torch.empty_like(x)
    w = torch.ones(64, device="cuda")
    rope = table(8, 64).cuda()
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")

    def code(heads, p=pos):
        with pytest.raises(ic.ICError) as e:
            ic.ic_qk_norm_rope(ctx, heads, p)
        return e.value.code

    assert code([], None) == ic.IC_ERR_SHAPE
    assert code([dict(x=x, out=o)] * 9) == ic.IC_ERR_SHAPE
    assert code([dict(x=x, out=o, weight=w)]) == ic.IC_ERR_INVALID_ARG
    assert code([dict(x=x, out=o, norm="rms", bias=w)]) == ic.IC_ERR_INVALID_ARG
    assert code([dict(x=x, out=o, norm="rms", eps=0.0)]) == ic.IC_ERR_SHAPE
    assert code([dict(x=x, out=o, norm="rms", eps=float("nan"))]) == ic.IC_ERR_SHAPE
    assert code([dict(x=x, out=o, rope=rope)], None) == ic.IC_ERR_INVALID_ARG
    assert code([dict(x=x, out=o, rope=table(8, 24).cuda())]) == ic.IC_ERR_UNSUPPORTED
    assert code([dict(x=x, out=o, rope=table(8, 80).cuda())]) == ic.IC_ERR_UNSUPPORTED
    x48 = torch.ones((4, 2, 48), dtype=torch.bfloat16, device="cuda")
    assert code([dict(x=x48, out=torch.empty_like(x48))]) == ic.IC_ERR_UNSUPPORTED
    odd = torch.ones((4, 2 * 64 + 4), dtype=torch.bfloat16, device="cuda")[:, :128].unflatten(1, (2, 64))
    assert code([dict(x=odd, out=o)]) == ic.IC_ERR_SHAPE
    skew = torch.ones(4 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(4, 2, 64)
    assert code([dict(x=skew, out=o)]) == ic.IC_ERR_INVALID_ARG
    # outputs on their inputs, or on each other
    assert code([dict(x=x, out=x)]) == ic.IC_ERR_INVALID_ARG
    assert code([dict(x=x, out=o), dict(x=x, out=o)]) == ic.IC_ERR_INVALID_ARG
    some = torch.arange(4, dtype=torch.int64, device="cuda")
    assert code([dict(x=x, out=o, slot=some), dict(x=x, out=o)]) == ic.IC_ERR_INVALID_ARG
    both = torch.zeros((8, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert code([dict(x=both[:4], out=both[3:7])]) == ic.IC_ERR_INVALID_ARG
    ic.ic_qk_norm_rope(ctx, [dict(x=both[:4], out=both[4:])])
    for heads in ([dict(x=x)], [dict(x=x, out=o, out8=o)], [dict(x=x, out=o[:3])],
                  [dict(x=x, out=o, weights=w)], [dict(x=x.transpose(0, 1), out=o)],
                  [dict(x=x, out=o), dict(x=x[:2], out=o[:2])]):
        with pytest.raises((ValueError, TypeError)):
            ic.ic_qk_norm_rope(ctx, heads, pos)
    with pytest.raises(TypeError):
        ic.ic_qk_norm_rope(ctx, [dict(x=x.half(), out=o)], pos)
    empty = torch.ones((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    ic.ic_qk_norm_rope(ctx, [dict(x=empty, out=torch.empty_like(empty))])
    ctx.sync_status()


def test_captured_and_on_another_stream(ic, ctx):
    """Captured once and replayed on new contents, launched on a stream of its own."""
    rows = 64
    x = torch.randn((rows, 4, 128), device="cuda").bfloat16()
    rope, pos = table(99, 128).cuda(), torch.arange(rows, dtype=torch.int32, device="cuda")
    o = torch.zeros_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ic.ic_qk_norm_rope(ctx, [dict(x=x, norm="rms", rope=rope, out=o)], pos)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        want = torch.zeros_like(x)
        ic.ic_qk_norm_rope(ctx, [dict(x=x, norm="rms", rope=rope, out=want)], pos)
        ctx.sync_status()
        assert torch.equal(o, want)
    assert np.isfinite(o.float().cpu().numpy()).all()
