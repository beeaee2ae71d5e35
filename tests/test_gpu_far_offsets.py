"""Drafted-token operators and norm + rotation on tensors whose elements lie more
than 2^31 elements or 2^32 bytes from their start."""
import math

import pytest
import torch

import tests.tree_ref as ref
from tests.test_gpu_norm_rope import check_bf16, check_fp8, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ic():
    from cross_layer_top_b200 import indexcache
    return indexcache


@pytest.fixture()
def ctx(ic):
    c = ic.Context(0)
    yield c
    c.close()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_of_a_long_tensor(ic, ctx, fp8):
    """3.4e9 values in, and out in reversed rows."""
    rows, H, d = 410_000, 64, 128
    assert rows * H * d > 2 ** 31 + 2 ** 30
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, H, d), dtype=torch.bfloat16, device="cuda")
    for c in x.split(50_000):
        c.copy_(torch.randn(c.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    rope = table(4096, d)
    pos = (torch.arange(rows, dtype=torch.int32) * 7) % 4096
    slot = torch.arange(rows - 1, -1, -1, device="cuda")
    head = dict(x=x, norm="rms", rope=rope.cuda(), slot=slot)
    if fp8:
        o, sc = torch.zeros((rows, H, d), dtype=torch.uint8, device="cuda"), torch.zeros((rows, H), device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out8=o, out_scale=sc)], pos.cuda())
    else:
        o = torch.zeros((rows, H, d), dtype=torch.bfloat16, device="cuda")
        ic.ic_qk_norm_rope(ctx, [dict(head, out=o)], pos.cuda())
    ctx.sync_status()
    at = torch.tensor([0, 1, 131_071, 131_072, 262_143, 262_144, 262_145, 393_216, rows - 2, rows - 1])
    z, tol = ref.norm_rope(x[at.cuda()].cpu(), "rms", None, None, 1e-6, rope, pos[at], False)
    to = (rows - 1 - at).cuda()
    if fp8:
        check_fp8(o[to].cpu(), sc[to].cpu(), z, tol)
        assert (sc > 0).all()
    else:
        check_bf16(o[to].cpu(), z, tol)
        assert o.view(torch.int32).ne(0).any(-1).all()


def test_scores_of_a_long_cache(ic, ctx):
    """4.6e9 bytes of keys: integer inputs, every score exact, at sampled keys of each sequence."""
    B, T, H, S = 3, 2, 64, 12_000_001
    assert B * S * 128 > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(2)
    k8 = torch.empty((B, S, 128), dtype=torch.uint8, device="cuda")
    code = torch.arange(-4, 5, device="cuda").float().to(torch.float8_e4m3fn).view(torch.uint8)
    for c in k8.view(-1, 128).split(2_000_000):
        c.copy_(code[torch.randint(0, 9, c.shape, generator=g, device="cuda", dtype=torch.uint8).int()])
    scale = torch.tensor([0.25, 1.0, 2.0], device="cuda")[
        torch.randint(0, 3, (B, S), generator=g, device="cuda")]
    q = torch.randint(-3, 4, (B, T, H, 128), generator=g, device="cuda").bfloat16()
    w = torch.tensor([-1.0, -0.5, 0.5, 1.0], device="cuda")[
        torch.randint(0, 4, (B, T, H), generator=g, device="cuda")].bfloat16()
    prefix = [S - T, S - 100, 11_999_000]
    ld = (S + 3) // 4 * 4
    out = torch.full((B * T, ld), 777.0, device="cuda")
    ic.ic_index_score_tree(ctx, q, w, k8, scale, torch.tensor(prefix, dtype=torch.int32, device="cuda"), out)
    ctx.sync_status()
    got = out.view(B, T, ld)
    for b in range(B):
        end = prefix[b] + T
        at = torch.cat([torch.arange(0, 300), torch.arange(end - 300, end),
                        torch.arange(8_388_000, 8_389_000)]).cuda()
        k = k8[b, at].view(torch.float8_e4m3fn).double()
        for t in range(T):
            want = (w[b, t].double() @ (q[b, t].double() @ k.T).clamp_min(0)) * scale[b, at].double()
            want[at > prefix[b] + t] = -math.inf
            assert torch.equal(got[b, t, at].double(), want), (b, t)
            assert (got[b, t, end:] == 777.0).all() and not (got[b, t, :end] == 777.0).all()


@pytest.mark.parametrize("listed", [False, True])
def test_attention_over_the_longest_cache(ic, ctx, listed):
    """Two sequences of 2^24 slots.  A few keys far from the start carry the weight: e^-20 is what
    all others could add."""
    B, T, Hq, d, S = 2, 3, 2, 128, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.empty((B, S, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (K, V):
        for c in t.view(-1, d).split(2_000_000):
            c.copy_(torch.randn(c.shape, generator=g, device="cuda", dtype=torch.bfloat16))
    K.mul_(1 / 64)
    Q = torch.randn((B, T, Hq, d), generator=g, device="cuda").bfloat16()
    prefix = [S - T, S - 777]
    spots = [5, (1 << 23) + 1, (1 << 24) - 1000, (1 << 24) - 900]
    # a component that the planted keys share with every query: logits of 60 apart from the rest
    Q[..., 0] = 30.0
    K[:, :, 0] = 0
    for i, s in enumerate(spots):
        K[:, s] = 0
        K[:, s, 0] = 2.0 - 0.03125 * i
    for b in range(B):  # drafts: of little weight, like the rest
        K[b, prefix[b]:prefix[b] + T, 0] = 0
    idx = None
    if listed:
        idx = torch.full((B, 300), -1, dtype=torch.int32, device="cuda")
        idx[:, ::2] = torch.arange(150, device="cuda", dtype=torch.int32) * 100_000 + 17
        idx[:, [0, 2, 100, 298]] = torch.tensor(spots, dtype=torch.int32, device="cuda")
    out = torch.zeros((B, T, Hq, d), dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q, K, V, torch.tensor(prefix, dtype=torch.int32, device="cuda"), out, idx=idx, scale=1.0)
    ctx.sync_status()
    at = torch.tensor(spots, device="cuda")
    for b in range(B):
        # every logit but those of the spots: below |q| |k| without the first component
        far = (Q[b, ..., 1:].double().norm(dim=-1).max() *
               torch.stack([c[:, 1:].float().norm(dim=-1).max() for c in K[b].split(2_000_000)]).max().double())
        z = Q[b].double() @ K[b, at].double().T
        assert float(z.min() - far) > math.log(S) + 20
        p = torch.softmax(z, -1)
        v = V[b, at].double()
        want = p @ v
        mean_abs = p @ v.abs()
        dz = (Q[b].double().abs() @ K[b, at].double().abs().T).amax(-1, keepdim=True) * (d + 4) * ref.U32T
        tol = want.abs() * ref.UBF16 + mean_abs * (ref.UBF16 * 1.01 + 2 * dz + 2.0 ** -21) + \
            math.exp(-20) * V[b, at].double().abs().max() * 8
        assert ((out[b].double() - want).abs() <= tol).all(), b
