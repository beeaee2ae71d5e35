"""Outputs of the drafted-token operators and of ic_qk_norm_rope on memory that
the same call reads, the small tensors (positions, lengths, masks, lists)
among it: refused before anything is launched, and nothing is written."""
import pytest
import torch

from tests.test_gpu_norm_rope import table

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


def refused(ic, ctx, call):
    with pytest.raises(ic.ICError) as e:
        call()
    assert e.value.code == ic.IC_ERR_INVALID_ARG and "overlap" in str(e.value)
    ctx.sync_status()


class Shared:
    """Zeroed bytes of which tensors are taken: the first of each pair of tensors overlaps the next."""

    def __init__(self, nbytes=1 << 20):
        self.bytes = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")

    def take(self, shape, dtype, at=0):
        n = torch.Size(shape).numel() * dtype.itemsize
        return self.bytes[at:at + n].view(dtype).view(shape)


# ---------------------------------------------------------- norm and rotation
@pytest.mark.parametrize("what", ["weight", "bias", "rope", "pos", "slot"])
@pytest.mark.parametrize("scale", [False, True])
def test_norm_rope_output_on_a_small_input(ic, ctx, what, scale):
    rows, H, d = 40, 1, 64
    x = torch.ones((rows, H, d), dtype=torch.bfloat16, device="cuda")
    m = Shared()
    head = dict(x=x, norm="layer", weight=torch.ones(d, device="cuda"), bias=torch.ones(d, device="cuda"),
                rope=table(8, d).cuda(), slot=torch.arange(rows, device="cuda"))
    pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
    at = 16 * rows if scale else 0  # somewhere inside
    if what == "pos":
        pos = m.take((rows,), torch.int32)
        at = 16 if scale else 0
    else:
        like = head[what]
        head[what] = m.take(like.shape, like.dtype)
        at = 16
    if scale:
        head.update(out8=torch.zeros((rows, H, d), dtype=torch.uint8, device="cuda"),
                    out_scale=m.take((rows, H), torch.float32, at))
    else:
        head.update(out=m.take((rows, H, d), torch.bfloat16, at))
    refused(ic, ctx, lambda: ic.ic_qk_norm_rope(ctx, [head], pos))
    other = dict(x=x, norm="rms", out=torch.zeros_like(x))  # the same from another tensor of the call
    refused(ic, ctx, lambda: ic.ic_qk_norm_rope(ctx, [other, head], pos))
    assert (m.bytes == 0).all()


def test_norm_rope_outputs_that_slots_do_not_tell_apart(ic, ctx):
    rows, H, d = 12, 2, 64
    x = torch.ones((rows, H, d), dtype=torch.bfloat16, device="cuda")
    one = torch.ones((rows, 1, d), dtype=torch.bfloat16, device="cuda")
    slot = torch.arange(rows, device="cuda")
    m = Shared()
    # its own scales on its own values
    refused(ic, ctx, lambda: ic.ic_qk_norm_rope(ctx, [
        dict(x=x, out8=m.take((rows, H, d), torch.uint8), out_scale=m.take((rows, H), torch.float32, 64),
             slot=slot)]))
    # rows of two sizes, and rows of one size half a row apart
    refused(ic, ctx, lambda: ic.ic_qk_norm_rope(ctx, [
        dict(x=x, out=m.take((30, H, d), torch.bfloat16), slot=slot),
        dict(x=one, out=m.take((30, 1, d), torch.bfloat16, 512), slot=slot + 12)]))
    refused(ic, ctx, lambda: ic.ic_qk_norm_rope(ctx, [
        dict(x=x, out=m.take((30, H, d), torch.bfloat16), slot=slot),
        dict(x=x, out=m.take((30, H, d), torch.bfloat16, 128), slot=slot + 15)]))
    assert (m.bytes == 0).all()
    # whole rows apart: the slots tell them apart
    a, b = m.take((30, H, d), torch.bfloat16), m.take((28, H, d), torch.bfloat16, 2 * H * d * 2)
    ic.ic_qk_norm_rope(ctx, [dict(x=x, out=a, slot=slot), dict(x=x * 2, out=b, slot=slot + 10)])
    ctx.sync_status()
    assert (a[:12] == 1).all() and (a[12:24] == 2).all() and (a[24:] == 0).all()


# ------------------------------------------------------------- drafted tokens
B, T, S = 2, 4, 64


def tree_tensors():
    p = torch.full((B,), 10, dtype=torch.int32, device="cuda")
    d = torch.full((B,), T, dtype=torch.int32, device="cuda")
    m = torch.ones((B, T), dtype=torch.int64, device="cuda")
    return dict(prefix=p, draft=d, mask=m)


@pytest.mark.parametrize("what", ["q", "w", "kI8", "kI_scale", "prefix", "draft", "mask"])
def test_tree_index_output_on_an_input(ic, ctx, what):
    H = 32
    m = Shared()
    t = dict(tree_tensors(), q=torch.zeros((B, T, H, 128), dtype=torch.bfloat16, device="cuda"),
             w=torch.zeros((B, T, H), dtype=torch.bfloat16, device="cuda"),
             kI8=torch.zeros((B, S, 128), dtype=torch.uint8, device="cuda"),
             kI_scale=torch.ones((B, S), device="cuda"))
    t[what] = m.take(t[what].shape, t[what].dtype, 64)
    args = [t[n] for n in ("q", "w", "kI8", "kI_scale", "prefix")]
    opt = dict(draft_len=t["draft"], tree_mask=t["mask"])
    scores, idx = m.take((B * T, S), torch.float32), m.take((B * T, 8), torch.int32)
    refused(ic, ctx, lambda: ic.ic_index_score_tree(ctx, *args, scores, **opt))
    refused(ic, ctx, lambda: ic.ic_index_fp_tree(ctx, *args, 8, idx, **opt))
    assert (m.bytes == 0).all()
    # right behind the input: nothing is shared
    ic.ic_index_score_tree(ctx, *args, m.take((B * T, S), torch.float32, 1 << 19), **opt)
    ctx.sync_status()


@pytest.mark.parametrize("what", ["Q", "K", "V", "prefix", "draft", "mask", "idx"])
def test_tree_attention_output_on_an_input(ic, ctx, what):
    Hq, d = 4, 64
    m = Shared()
    t = dict(tree_tensors(), Q=torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda"),
             K=torch.zeros((B, S, d), dtype=torch.bfloat16, device="cuda"),
             V=torch.zeros((B, S, d), dtype=torch.bfloat16, device="cuda"),
             idx=torch.full((B, 6), -1, dtype=torch.int32, device="cuda"))  # prefix may be 0
    t[what] = m.take(t[what].shape, t[what].dtype, 64)
    args = [t[n] for n in ("Q", "K", "V", "prefix")]
    opt = dict(draft_len=t["draft"], tree_mask=t["mask"], idx=t["idx"])
    refused(ic, ctx, lambda: ic.ic_tree_attn(ctx, *args, m.take((B, T, Hq, d), torch.bfloat16), **opt))
    assert (m.bytes == 0).all()
    ic.ic_tree_attn(ctx, *args, m.take((B, T, Hq, d), torch.bfloat16, 1 << 19), **opt)
    ctx.sync_status()
