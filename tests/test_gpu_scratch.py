"""The context's scratch buffers while graphs hold their addresses: what must
not move is refused, and nothing else is."""
import pytest
import torch

import tests.tree_ref as ref
from cross_layer_top_b200 import synth

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


def decode_inputs(B, S, seed=1):
    """q, w, kI8, kI_scale of one new token a sequence, small integers (scores are exact)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-3, 4, (B, 64, 128), generator=g).bfloat16()
    w = torch.tensor([-1.0, -0.5, 0.5, 1.0])[torch.randint(0, 4, (B, 64), generator=g)].bfloat16()
    k8 = torch.randint(-4, 5, (B, S, 128), generator=g).float().to(torch.float8_e4m3fn)
    return q.cuda(), w.cuda(), k8.view(torch.uint8).cuda(), torch.ones((B, S), device="cuda")


def decode_stack(ic, B=2, S=2500):
    cfg = synth.DecodeConfig("held", B, S, "FS", 64, 128, 256, 16, 128, 3)
    layers = []
    for ell in range(cfg.n_layers):
        lay = synth.decode_layer(cfg, ell, "cuda")
        lay["out"] = torch.zeros((B, cfg.Hq, cfg.d), dtype=torch.bfloat16, device="cuda")
        layers.append(lay)
    dims = ic.stack_dims(ic.IC_DECODE, cfg.H_I, cfg.d_I, cfg.k, cfg.Hq, cfg.d, B=B, S_max=S,
                         seq_len=layers[0]["seq_len"])
    return layers, dims, torch.zeros((B, cfg.k), dtype=torch.int32, device="cuda")


def stack_graph(ic, ctx):
    """A decode stack's graph on ctx, its attention outputs and index cache."""
    layers, dims, cache = decode_stack(ic)
    g = ic.ic_stack_graph_create(ctx, ic.ic_create_pattern("FS"), layers, dims, cache)
    return g, [lay["out"] for lay in layers], cache


def replayed(g, outs, cache):
    for t in outs + [cache]:
        t.zero_()
    g.launch()
    torch.cuda.synchronize()
    return [t.clone() for t in outs + [cache]]


@pytest.mark.parametrize("ahead", [False, True])
def test_a_stack_graph_waits_for_the_work_before_it(ic, ctx, ahead):
    """Its eager pass shares the index buffer and the scratch with the caller's streams: what they
    hold at the call comes first."""
    layers, dims, cache = decode_stack(ic)
    more = [torch.zeros_like(cache)] if ahead else []
    create = ic.ic_stack_graph_create_ahead if ahead else ic.ic_stack_graph_create
    for _ in range(2):  # the first one loads kernels and allocates, which waits by itself
        torch.cuda._sleep(200_000_000)  # about 0.1 s
        cache.fill_(-9)
        g = create(ctx, ic.ic_create_pattern("FS"), layers, dims, cache, *more)
        ctx.sync_status()
        assert (cache >= 0).all()
        g.close()


def test_first_tree_attention_beside_a_stack_graph(ic, ctx):
    """No graph can hold a workspace that is not there yet: the first call allocates it, and the
    graph replays as before."""
    g, outs, cache = stack_graph(ic, ctx)
    before = replayed(g, outs, cache)
    gen = torch.Generator().manual_seed(2)
    Q = torch.randn((2, 3, 4, 64), generator=gen).bfloat16()
    K, V = (torch.randn((2, 90, 64), generator=gen).bfloat16() for _ in range(2))
    out = torch.zeros(Q.shape, dtype=torch.bfloat16, device="cuda")
    ic.ic_tree_attn(ctx, Q.cuda(), K.cuda(), V.cuda(), torch.tensor([80, 5], dtype=torch.int32).cuda(), out)
    ctx.sync_status()
    for b, n in enumerate((80, 5)):
        want, tol = ref.tree_attn(Q[b], K[b], V[b], n, 3, None, None, 0.125)
        assert ((out[b].cpu().double() - want).abs() <= tol).all()
    assert all(torch.equal(a, b) for a, b in zip(before, replayed(g, outs, cache)))
    ctx.sync_status()
    g.close()


def tree_call(ic, ctx, B, T, S, k=64, seed=3):
    """ic_index_fp_tree's arguments and the call, its index rows first."""
    q, w, k8, scale = decode_inputs(B, S, seed)
    q, w = (t.repeat_interleave(T, 0).view(B, T, *t.shape[1:]).contiguous() for t in (q, w))
    prefix = torch.full((B,), S - T, dtype=torch.int32, device="cuda")
    idx = torch.zeros((B * T, k), dtype=torch.int32, device="cuda")
    return idx, lambda c=ctx: ic.ic_index_fp_tree(c, q, w, k8, scale, prefix, k, idx)


def decode_call(ic, ctx, B, S, k=64, seed=4):
    q, w, k8, scale = decode_inputs(B, S, seed)
    seq = torch.full((B,), S, dtype=torch.int32, device="cuda")
    idx = torch.zeros((B, k), dtype=torch.int32, device="cuda")
    return idx, lambda c=ctx: ic.ic_index_fp_decode(c, q, w, k8, scale, seq, k, idx)


def prefill_call(ic, ctx, L, k=64):
    g = torch.Generator().manual_seed(6)
    qI, kI, w = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((L, 64, 128), (L, 128), (L, 64)))
    idx = torch.zeros((L, k), dtype=torch.int32, device="cuda")
    return idx, lambda c=ctx: ic.ic_index_fp(c, qI, kI, w, k, idx)


def captured(call):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        call()
    return graph


def replay(graph, idx):
    idx.zero_()
    graph.replay()
    torch.cuda.synchronize()
    return idx.clone()


def elsewhere(ic, idx, call):
    """What the call gives in a context of its own."""
    idx.zero_()
    c = ic.Context(0)
    call(c)
    c.sync_status()
    c.close()
    return idx.clone()


def refused(ic, call):
    with pytest.raises(ic.ICError) as e:
        call()
    assert e.value.code == ic.IC_ERR_NOMEM and "captured" in str(e.value)


def test_a_capture_holds_no_more_than_its_own_buffers(ic, ctx):
    """A captured ic_index_fp_tree holds the score rows; the decode step's histograms, which it does
    not use, still grow."""
    decode_call(ic, ctx, 1, 17000)[1]()  # histograms of one sequence
    idx, call = tree_call(ic, ctx, 2, 8, 17000)
    call()
    want = idx.clone()
    graph = captured(call)
    idx4, call4 = decode_call(ic, ctx, 4, 17000)  # its score rows fit, its histograms do not
    call4()
    ctx.sync_status()
    got = idx4.clone()
    assert torch.equal(got, elsewhere(ic, idx4, call4))
    assert torch.equal(replay(graph, idx), want)
    ctx.sync_status()
    del graph


def test_scratch_grows_again_when_the_graph_is_gone(ic, ctx):
    idx, call = tree_call(ic, ctx, 2, 2, 500)
    call()
    graph = captured(call)
    idx2, bigger = tree_call(ic, ctx, 2, 4, 3000)
    refused(ic, bigger)
    del graph
    bigger()
    ctx.sync_status()
    got = idx2.clone()
    assert torch.equal(got, elsewhere(ic, idx2, bigger))


@pytest.mark.parametrize("what", ["decode", "prefill", "stack"])
def test_captured_calls_keep_their_scratch(ic, ctx, what):
    """A user's graph of a call that scores through the context's scratch: a call that would move it is
    refused while the graph lives, and the graph replays the same indices."""
    if what == "decode":
        idx, call = decode_call(ic, ctx, 2, 2500)
    elif what == "prefill":
        idx, call = prefill_call(ic, ctx, 300)
    else:
        layers, dims, idx = decode_stack(ic)
        pattern = ic.ic_create_pattern("FS")
        call = lambda: ic.ic_run_stack(ctx, pattern, layers, dims, idx)  # noqa: E731
    call()
    ctx.sync_status()
    want = idx.clone()
    graph = captured(call)
    idx2, bigger = tree_call(ic, ctx, 4, 8, 3000)
    refused(ic, bigger)
    assert torch.equal(replay(graph, idx), want)
    ctx.sync_status()
    del graph
    bigger()
    ctx.sync_status()


def test_captured_decode_keeps_its_histograms(ic, ctx):
    tree_call(ic, ctx, 2, 8, 17000)[1]()  # score rows for all that follows
    idx, call = decode_call(ic, ctx, 1, 17000)
    call()
    want = idx.clone()
    graph = captured(call)
    idx4, more = decode_call(ic, ctx, 4, 17000)
    refused(ic, more)
    assert torch.equal(replay(graph, idx), want)
    del graph
    more()
    ctx.sync_status()
    got = idx4.clone()
    assert torch.equal(got, elsewhere(ic, idx4, more))


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_first_call_inside_a_capture_leaves_it_alive(ic, ctx, what):
    idx, call = decode_call(ic, ctx, 2, 2500) if what == "decode" else prefill_call(ic, ctx, 300)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        idx.fill_(7)
        with pytest.raises(ic.ICError) as e:
            call()
        assert e.value.code == ic.IC_ERR_NOMEM and "capture" in str(e.value)
    assert (replay(graph, idx) == 7).all()
    call()
    ctx.sync_status()
    assert not (idx == 7).all()


def test_stack_graph_holds_what_it_uses(ic, ctx):
    """A stack graph of short sequences uses no histograms: those of another call may grow beside it,
    its score rows may not; a destroyed graph holds nothing."""
    tree_call(ic, ctx, 2, 8, 17000)[1]()  # score rows for the decode calls
    decode_call(ic, ctx, 1, 17000)[1]()
    g, outs, cache = stack_graph(ic, ctx)
    before = replayed(g, outs, cache)
    decode_call(ic, ctx, 4, 17000)[1]()
    idx, bigger = tree_call(ic, ctx, 4, 8, 17000)
    with pytest.raises(ic.ICError) as e:
        bigger()
    assert e.value.code == ic.IC_ERR_NOMEM
    assert all(torch.equal(a, b) for a, b in zip(before, replayed(g, outs, cache)))
    ctx.sync_status()
    g.close()
    bigger()
    ctx.sync_status()
