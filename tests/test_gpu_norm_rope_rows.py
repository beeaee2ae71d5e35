"""ic_qk_norm_rope on tensors of many heads, whose warps take whole chunks of
one row: every vector size, slots, errors and rows far enough apart that a
warp prefetches a later one's values.  Bounds from tests/tree_ref.py."""
import pytest
import torch

import tests.tree_ref as ref
from tests.test_gpu_norm_rope import check_bf16, check_fp8, table

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


# rows, H, d, d_rot, norm, interleaved, fp8
CASES = [(37, 16, 64, 64, "rms", False, False), (37, 16, 64, 32, "layer", True, True),
         (41, 32, 32, 32, "rms", False, True), (41, 64, 32, 16, "layer", True, False),
         (53, 8, 128, 128, "rms", True, False), (53, 8, 128, 64, None, False, True),
         (29, 16, 128, 128, "layer", False, False), (29, 48, 128, 0, "layer", False, True),
         (19, 64, 64, 48, None, True, False)]


@pytest.mark.parametrize("rows,H,d,dr,norm,inter,fp8", CASES)
def test_many_heads_at_slots(ic, ctx, rows, H, d, dr, norm, inter, fp8):
    """Permuted slots, -1 among them: rows go where they are told, all others keep their bytes."""
    g = torch.Generator().manual_seed(rows * H + d)
    base = (torch.randn((rows, H * d + 16), generator=g) * 2 + 0.3).bfloat16()
    x, xg = base[:, 8:8 + H * d].unflatten(1, (H, d)), base.cuda()[:, 8:8 + H * d].unflatten(1, (H, d))
    wt = 1 + 0.2 * torch.randn(d, generator=g) if norm else None
    bs = 0.2 * torch.randn(d, generator=g) if norm == "layer" else None
    rope = table(900, dr) if dr else None
    pos = torch.randint(0, 900, (rows,), generator=g, dtype=torch.int32)
    cache = rows + 11
    slot = torch.randperm(cache, generator=g)[:rows]
    slot[::5] = -1
    z, tol = ref.norm_rope(x, norm, wt, bs, 1e-6, rope, pos, inter)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    head = dict(x=xg, norm=norm, weight=cu(wt), bias=cu(bs), rope=cu(rope), interleaved=inter, slot=slot.cuda())
    live = slot >= 0
    rest = torch.ones(cache, dtype=torch.bool)
    rest[slot[live]] = False
    if fp8:
        o = torch.full((cache, H, d), 0x55, dtype=torch.uint8, device="cuda")
        sc = torch.full((cache, H), -1.0, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out8=o, out_scale=sc)], pos.cuda())
        ctx.sync_status()
        o, sc = o.cpu(), sc.cpu()
        check_fp8(o[slot[live]], sc[slot[live]], z[live], tol[live])
        assert (o[rest] == 0x55).all() and (sc[rest] == -1).all()
    else:
        o = torch.full((cache, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out=o)], pos.cuda())
        ctx.sync_status()
        o = o.cpu()
        check_bf16(o[slot[live]], z[live], tol[live])
        assert (o[rest] == 9.0).all()


@pytest.mark.parametrize("H,d", [(16, 64), (32, 32), (8, 128), (64, 128)])
def test_a_bad_row_of_many_heads_is_reported_and_left_out(ic, ctx, H, d):
    rows = 23
    x = torch.ones((rows, H, d), dtype=torch.bfloat16, device="cuda")
    rope = table(50, d).cuda()
    for bad_pos, bad_slot in ((50, None), (-1, None), (None, -2), (None, 40)):
        pos, slot = torch.full((rows,), 3, dtype=torch.int32), torch.arange(rows)
        if bad_pos is None:
            slot[13] = bad_slot
        else:
            pos[13] = bad_pos
        o = torch.full((40, H, d), 9.0, dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(x=x, rope=rope, out=o, slot=slot.cuda())], pos.cuda())
        with pytest.raises(ic.ICError) as e:
            ctx.sync_status()
        assert e.value.code == ic.IC_ERR_DEVICE and ("slot" if bad_pos is None else "position") in str(e.value)
        kept = (o == 9.0).flatten(1).all(1).cpu()
        assert kept[13] and kept[rows:].all() and kept.sum() == 1 + 40 - rows


@pytest.mark.parametrize("rows,H,fp8", [(2003, 64, False), (2003, 64, True), (7001, 16, False)])
def test_rows_far_ahead_are_prefetched(ic, ctx, rows, H, fp8):
    """More vectors than a quarter of the resident warps hold: values of later warps are asked for on
    the way, up to the tensor's last row (strided, the end of its memory right behind it)."""
    d = 128
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 22 // 4
    assert rows * H > 2 * warps * 32
    g = torch.Generator().manual_seed(rows)
    base = torch.randn((rows, H * d + 8), generator=g).bfloat16()
    xg = base.cuda().flatten()[8:].as_strided((rows, H, d), (H * d + 8, d, 1))
    x = base[:, 8:].unflatten(1, (H, d))
    rope, pos = table(4096, d), torch.randint(0, 4096, (rows,), generator=g, dtype=torch.int32)
    z, tol = ref.norm_rope(x, "rms", None, None, 1e-6, rope, pos, False)
    head = dict(x=xg, norm="rms", rope=rope.cuda())
    if fp8:
        o, sc = torch.zeros((rows, H, d), dtype=torch.uint8, device="cuda"), torch.zeros((rows, H), device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out8=o, out_scale=sc)], pos.cuda())
        ctx.sync_status()
        check_fp8(o.cpu(), sc.cpu(), z, tol)
    else:
        o = torch.zeros((rows, H, d), dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out=o)], pos.cuda())
        ctx.sync_status()
        check_bf16(o.cpu(), z, tol)
