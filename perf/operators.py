"""The operators of a drafted-token step, as they are measured.

One step of the sparse-attention path over several new tokens per sequence:
``norm_rope`` turns projected rows into queries, cache rows and FP8 indexer
keys (per-head norm, position rotation, quantisation, cache write);
``tree_score`` scores the drafted tokens' indexer queries against the FP8
indexer-key cache; ``tree_attn`` attends from the drafted tokens to the
cached prefix (all of it, or one shared list of selected positions) and to
their own ancestors.

``run`` computes the plain form in elementary torch operations, or, where
``own`` is true, calls the library.
"""
import math

import torch

own = False

_F32 = torch.float32
_BF16 = torch.bfloat16
_ctx = None


# --------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of a small batch (drafts of two per sequence, some
        # rows padding): Q, K, V, q_I and k_I of every new token
        dict(name="rope_decode", op="norm_rope", rows=64, hq=16, d=128, hi=64, di=128, drot=128,
             dirot=64, q8=False, inter=False, cache=4096, pad=5),
        # a prompt of the prefill workload's length, FP8 queries too
        dict(name="rope_prompt", op="norm_rope", rows=16384, hq=16, d=128, hi=64, di=128,
             drot=128, dirot=64, q8=True, inter=False, cache=16384, pad=0),
        # the small model's heads, an odd number of rows, rotation by pairs
        dict(name="rope_small", op="norm_rope", rows=511, hq=4, d=64, hi=4, di=32, drot=32,
             dirot=32, q8=True, inter=True, cache=700, pad=3),
        # the least: one token of one sequence, a short context
        dict(name="score_one", op="tree_score", b=1, t=1, hi=64, s=777, draft_pad=False),
        # four drafts each at the batched decode workload's cache
        dict(name="score_batch", op="tree_score", b=32, t=4, hi=64, s=65537, draft_pad=False),
        # a wide tree at the long-context workload's cache
        dict(name="score_long", op="tree_score", b=8, t=16, hi=64, s=200001, draft_pad=False),
        # ragged: fewer heads, odd sizes, padded drafts
        dict(name="score_ragged", op="tree_score", b=3, t=13, hi=32, s=16421, draft_pad=True),
        # the least: a few drafts of one short sequence, the small heads
        dict(name="attn_one", op="tree_attn", b=1, t=3, hq=4, d=64, s=333, k=0, draft_pad=False),
        # eight drafts each at the long-context workload's cache, all of it
        dict(name="attn_long", op="tree_attn", b=8, t=8, hq=16, d=128, s=200001, k=0,
             draft_pad=False),
        # the widest tree over a prompt of the prefill workload's length
        dict(name="attn_wide", op="tree_attn", b=4, t=64, hq=16, d=128, s=16421, k=0,
             draft_pad=False),
        # selected positions, one list per sequence, at the batched decode
        # workload's cache
        dict(name="attn_list", op="tree_attn", b=32, t=8, hq=16, d=128, s=65537, k=2048,
             draft_pad=False),
        # ragged: odd everything, padded drafts, short list
        dict(name="attn_ragged", op="tree_attn", b=5, t=11, hq=7, d=64, s=9001, k=517,
             draft_pad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "tree_score", "tree_attn"])
    if op == "norm_rope":
        d, di = rng.choice([64, 128]), rng.choice([32, 64, 128])
        rows = _log_int(rng, 1, 16384)
        return dict(op=op, rows=rows, hq=rng.randint(1, 16), d=d, hi=rng.choice([4, 16, 32, 64]),
                    di=di, drot=rng.choice([d // 2, d]), dirot=rng.choice([di // 2, di]),
                    q8=rng.random() < 0.5, inter=rng.random() < 0.5,
                    cache=rows + rng.randint(1, 4096), pad=rng.randint(0, min(8, rows - 1)))
    t = _log_int(rng, 1, 64)
    s = _log_int(rng, 100, 200001)
    if op == "tree_score":
        hi = rng.choice([32, 64])
        most = 8 * 16 * 200001 * 64 // (t * s * hi)  # no more than the wide tree above
        while most < 1:
            s, most = s // 2, most * 2 or 1
        return dict(op=op, b=_log_int(rng, 1, min(32, most)), t=t, hi=hi, s=max(s, t + 1),
                    draft_pad=rng.random() < 0.5)
    hq, d = rng.randint(1, 16), rng.choice([64, 128])
    k = rng.choice([0, _log_int(rng, 16, 2048)])
    most = min(8 * 200001 // s, 4 * 64 * 16 * 16421 // (t * hq * (k or s)))
    while most < 1:
        s = s // 2
        most = min(8 * 200001 // s, 4 * 64 * 16 * 16421 // (t * hq * (k or s)))
    return dict(op=op, b=_log_int(rng, 1, min(32, most)), t=t, hq=hq, d=d, s=max(s, t + 1), k=k,
                draft_pad=rng.random() < 0.3)


# ---------------------------------------------------------------- the inputs
def _rope_table(n_pos, d_rot):
    """cos and sin of every position's angles, from 64 bits: [n_pos, d_rot]."""
    freq = 10000.0 ** (-torch.arange(0, d_rot, 2, dtype=torch.float64, device="cuda") / d_rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], dim=1).to(_F32).contiguous()


def _prepare_norm_rope(c, g):
    n, hq, d, hi, di = c["rows"], c["hq"], c["d"], c["hi"], c["di"]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # the projections' output as it lies in memory: one row per token that
    # holds every head of Q, K and V, another with those of q_I and k_I
    qkv = (rnd(n, (hq + 2) * d) * 2.0).to(_BF16)
    iqk = (rnd(n, (hi + 1) * di) * 1.5 + 0.1).to(_BF16)
    n_pos = 65536
    pos = torch.randint(0, n_pos, (n,), generator=g, device="cuda", dtype=torch.int32)
    # distinct cache rows; padding rows write none
    slot = torch.randperm(c["cache"], generator=g, device="cuda")[:n].to(torch.int64)
    if c["pad"]:
        slot[-c["pad"]:] = -1
    cache = c["cache"]
    st = dict(
        case=c, pos=pos, slot=slot,
        q=qkv[:, :hq * d].unflatten(1, (hq, d)), k=qkv[:, hq * d:(hq + 1) * d].unflatten(1, (1, d)),
        v=qkv[:, (hq + 1) * d:].unflatten(1, (1, d)),
        qI=iqk[:, :hi * di].unflatten(1, (hi, di)), kI=iqk[:, hi * di:].unflatten(1, (1, di)),
        q_weight=1 + 0.1 * rnd(d), k_weight=1 + 0.1 * rnd(d),
        kI_weight=1 + 0.1 * rnd(di), kI_bias=0.1 * rnd(di),
        rope=_rope_table(n_pos, c["drot"]), ropeI=_rope_table(n_pos, c["dirot"]),
        Q=torch.zeros((n, hq, d), dtype=_BF16, device="cuda"),
        K=rnd(cache, 1, d).to(_BF16), V=rnd(cache, 1, d).to(_BF16),
        kI8=torch.zeros((cache, 1, di), dtype=torch.uint8, device="cuda"),
        kI_scale=torch.ones((cache, 1), device="cuda"))
    if c["q8"]:
        st["qI8"] = torch.zeros((n, hi, di), dtype=torch.uint8, device="cuda")
        st["qI_scale"] = torch.ones((n, hi), device="cuda")
    else:
        st["qIr"] = torch.zeros((n, hi, di), dtype=_BF16, device="cuda")
    return st


def _trees(c, g):
    """Ragged prefixes and drafted trees: prefix_len, draft_len, mask of ancestors (and self)."""
    b, t, s = c["b"], c["t"], c["s"]
    low = max(0, s - t - max(1, s // 8))
    prefix = torch.randint(low, s - t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    prefix[0] = s - t
    draft = torch.full((b,), t, dtype=torch.int32, device="cuda")
    if c["draft_pad"]:
        draft = torch.randint(1, t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    up = (torch.rand((b, t), generator=g, device="cuda") *
          torch.arange(t, device="cuda")).to(torch.int64).cpu()
    mask = torch.zeros((b, t), dtype=torch.int64)
    for u in range(t):  # a node sees itself and what its parent sees
        mask[:, u] = 1 << u if u < 63 else -(1 << 63)
        if u:
            mask[:, u] |= mask.gather(1, up[:, u:u + 1])[:, 0]
    return prefix, draft, mask.cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "norm_rope":
        return _prepare_norm_rope(case, g)
    b, t, s = case["b"], case["t"], case["s"]
    prefix, draft, mask = _trees(case, g)
    st = dict(case=case, prefix=prefix, draft=draft, mask=mask)
    if case["op"] == "tree_score":
        hi = case["hi"]
        st["q"] = torch.randn((b, t, hi, 128), generator=g, device="cuda").to(_BF16)
        st["w"] = (torch.randn((b, t, hi), generator=g, device="cuda") / math.sqrt(hi)).to(_BF16)
        k = torch.randn((b, s, 128), generator=g, device="cuda")
        scale = k.abs().amax(-1) / 448.0
        st["kI8"] = (k / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st["kI_scale"] = scale
        st["scores"] = torch.zeros((b * t, (s + 63) // 64 * 64), device="cuda")
        return st
    hq, d, k = case["hq"], case["d"], case["k"]
    st["Q"] = torch.randn((b, t, hq, d), generator=g, device="cuda").to(_BF16)
    st["K"] = torch.randn((b, s, d), generator=g, device="cuda", dtype=_BF16)
    st["V"] = torch.randn((b, s, d), generator=g, device="cuda", dtype=_BF16)
    st["out"] = torch.zeros((b, t, hq, d), dtype=_BF16, device="cuda")
    st["idx"] = None
    if k:
        # ascending selected positions of the prefix, -1 behind the last
        r = torch.rand((b, s), generator=g, device="cuda")
        r.masked_fill_(torch.arange(s, device="cuda") >= prefix[:, None], -1.0)
        top = r.topk(min(k, s), dim=1)
        pos = torch.where(top.values >= 0, top.indices, s).sort(1).values
        idx = torch.full((b, k), -1, dtype=torch.int32, device="cuda")
        idx[:, :pos.shape[1]] = torch.where(pos < s, pos, -1).to(torch.int32)
        st["idx"] = idx
    return st


# -------------------------------------------------------------------- a pass
def _context():
    global _ctx
    from cross_layer_top_b200 import indexcache as ic
    if _ctx is None:
        _ctx = ic.Context(0)
    return ic, _ctx


def _rotate(y, cs, inter):
    """Rotate the first d_rot values of each head: pairs (i, i + d_rot/2), or (2i, 2i + 1)."""
    h = cs.shape[-1] // 2
    cos, sin, rot, rest = cs[:, None, :h], cs[:, None, h:], y[..., :2 * h], y[..., 2 * h:]
    if inter:
        a, b = rot[..., 0::2], rot[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :h], rot[..., h:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([out, rest], dim=-1)


def _rms(x, weight, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _layer_norm(x, weight, bias, eps):
    c = x - x.mean(-1, keepdim=True)
    return c * torch.rsqrt((c * c).mean(-1, keepdim=True) + eps) * weight + bias


def _fp8(y):
    scale = y.abs().amax(-1).clamp_min(1e-12) / 448.0
    return (y / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _norm_rope_outputs(st):
    out = dict(Q=st["Q"], K=st["K"], V=st["V"], kI8=st["kI8"].view(torch.float8_e4m3fn),
               kI_scale=st["kI_scale"])
    if st["case"]["q8"]:
        return out | dict(qI8=st["qI8"].view(torch.float8_e4m3fn), qI_scale=st["qI_scale"])
    return out | dict(qI=st["qIr"])


def _run_norm_rope(st):
    c, inter = st["case"], st["case"]["inter"]
    if own:
        ic, ctx = _context()
        heads = [dict(x=st["q"], norm="rms", weight=st["q_weight"], eps=1e-6, rope=st["rope"],
                      interleaved=inter, out=st["Q"]),
                 dict(x=st["k"], norm="rms", weight=st["k_weight"], eps=1e-6, rope=st["rope"],
                      interleaved=inter, out=st["K"], slot=st["slot"]),
                 dict(x=st["v"], out=st["V"], slot=st["slot"]),
                 dict(x=st["kI"], norm="layer", weight=st["kI_weight"], bias=st["kI_bias"],
                      eps=1e-6, rope=st["ropeI"], interleaved=inter, out8=st["kI8"],
                      out_scale=st["kI_scale"], slot=st["slot"])]
        if c["q8"]:
            heads.append(dict(x=st["qI"], rope=st["ropeI"], interleaved=inter, out8=st["qI8"],
                              out_scale=st["qI_scale"]))
        else:
            heads.append(dict(x=st["qI"], rope=st["ropeI"], interleaved=inter, out=st["qIr"]))
        ic.ic_qk_norm_rope(ctx, heads, st["pos"])
        return _norm_rope_outputs(st)
    at = st["pos"].to(torch.int64)
    cs, csI = st["rope"][at], st["ropeI"][at]
    live = st["slot"] >= 0
    slot = st["slot"][live]  # padding rows write no cache row
    st["Q"].copy_(_rotate(_rms(st["q"].to(_F32), st["q_weight"], 1e-6), cs, inter))
    st["K"][slot] = _rotate(_rms(st["k"].to(_F32), st["k_weight"], 1e-6), cs, inter)[live].to(_BF16)
    st["V"][slot] = st["v"][live]
    k8, scale = _fp8(_rotate(_layer_norm(st["kI"].to(_F32), st["kI_weight"], st["kI_bias"], 1e-6),
                             csI, inter))
    st["kI8"][slot] = k8[live]
    st["kI_scale"][slot] = scale[live]
    qI = _rotate(st["qI"].to(_F32), csI, inter)
    if c["q8"]:
        q8, scale = _fp8(qI)
        st["qI8"].copy_(q8)
        st["qI_scale"].copy_(scale)
    else:
        st["qIr"].copy_(qI)
    return _norm_rope_outputs(st)


def _sees(mask, prefix, draft, s):
    """[B, T, S]: whether row (b, t) sees cache slot s of its own sequence's drafts, and [B, S] of the prefix."""
    at = torch.arange(s, device=prefix.device)
    u = at[None, :] - prefix[:, None]
    drafted = (u >= 0) & (u < draft[:, None])
    bit = (mask[:, :, None] >> u.clamp(0, 63)[:, None, :]) & 1
    return drafted[:, None, :] & (bit != 0), u < 0


def _run_tree_score(st):
    if own:
        ic, ctx = _context()
        ic.ic_index_score_tree(ctx, st["q"], st["w"], st["kI8"], st["kI_scale"], st["prefix"],
                               st["scores"], draft_len=st["draft"], tree_mask=st["mask"])
        return st["scores"]
    c = st["case"]
    b, t, hi, s = c["b"], c["t"], c["hi"], c["s"]
    k = st["kI8"].view(torch.float8_e4m3fn).to(_F32) * st["kI_scale"][..., None]
    dots = torch.bmm(st["q"].to(_F32).reshape(b, t * hi, 128), k.transpose(1, 2))
    dots = dots.clamp_min_(0).mul_(st["w"].to(_F32).reshape(b, t * hi, 1))
    score = dots.view(b, t, hi, s).sum(2)
    seen, prefix = _sees(st["mask"], st["prefix"], st["draft"], s)
    score = torch.where(seen | prefix[:, None, :], score, -math.inf)
    live = torch.arange(t, device="cuda") < st["draft"][:, None]
    end = torch.arange(s, device="cuda") < (st["prefix"] + st["draft"])[:, None]
    old = st["scores"].view(b, t, -1)[:, :, :s]
    old.copy_(torch.where(live[:, :, None] & end[:, None, :], score, old))
    return st["scores"]


def _run_tree_attn(st):
    if own:
        ic, ctx = _context()
        ic.ic_tree_attn(ctx, st["Q"], st["K"], st["V"], st["prefix"], st["out"], idx=st["idx"],
                        draft_len=st["draft"], tree_mask=st["mask"])
        return st["out"]
    c = st["case"]
    b, t, hq, d, s = c["b"], c["t"], c["hq"], c["d"], c["s"]
    seen, prefix = _sees(st["mask"], st["prefix"], st["draft"], s)
    if st["idx"] is None:
        k, v, see = st["K"].to(_F32), st["V"].to(_F32), seen | prefix[:, None, :]
    else:
        # the listed prefix rows, then the drafted slots
        drafts = st["prefix"][:, None].to(torch.int64) + torch.arange(t, device="cuda")
        at = torch.cat([st["idx"].to(torch.int64), drafts], dim=1)
        listed_ = (st["idx"] >= 0)[:, None, :].expand(b, t, -1)
        at0 = at.clamp_min(0)
        see = torch.cat([listed_, seen.gather(2, drafts[:, None, :].expand(b, t, t))], dim=2)
        k = st["K"].gather(1, at0[:, :, None].expand(-1, -1, d)).to(_F32)
        v = st["V"].gather(1, at0[:, :, None].expand(-1, -1, d)).to(_F32)
    logits = torch.bmm(st["Q"].to(_F32).reshape(b, t * hq, d), k.transpose(1, 2))
    logits = logits.mul_(1.0 / math.sqrt(d)).view(b, t, hq, -1)
    logits.masked_fill_(~see[:, :, None, :], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = logits.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(b, t * hq, -1), v).view(b, t, hq, d)
    o = torch.where(total > 0, o / total, 0.0)
    live = torch.arange(t, device="cuda") < st["draft"][:, None]
    st["out"].copy_(torch.where(live[:, :, None, None], o, st["out"].to(_F32)))
    return st["out"]


_RUN = {"norm_rope": _run_norm_rope, "tree_score": _run_tree_score, "tree_attn": _run_tree_attn}


def run(state):
    return _RUN[state["case"]["op"]](state)


# ----------------------------------------------------------- what it cannot do without
def work(case):
    if case["op"] == "norm_rope":
        n, hq, d, hi, di = (case[k] for k in ("rows", "hq", "d", "hi", "di"))
        live = n - case["pad"]
        read = n * (hq * d + hi * di) * 2 + live * (2 * d + di) * 2 + n * 4 + live * 8
        read += n * (case["drot"] + case["dirot"]) * 4  # the positions' table rows
        wrote = n * hq * d * 2 + live * (2 * d * 2 + di + 4)
        wrote += n * hi * (di + 4) if case["q8"] else n * hi * di * 2
        return {"bytes": read + wrote, "flops": 10 * n * (hq * d + hi * di)}
    b, t, s = case["b"], case["t"], case["s"]
    # prefixes lie between 7/8 of the cache and all of it, and drafts fill half where they are padded
    mean_s = (s - t + (b - 1) * max(0, s - t - max(1, s // 8) / 2)) / b
    mean_t = (t + 1) / 2 if case["draft_pad"] else t
    if case["op"] == "tree_score":
        pairs = b * mean_t * (mean_s + mean_t)
        return {"bytes": b * (mean_s + mean_t) * 132 + b * mean_t * case["hi"] * 258 + pairs * 4,
                "flops": pairs * case["hi"] * 128 * 2}
    keys = (case["k"] if case["k"] else mean_s) + mean_t
    return {"bytes": b * (keys * case["d"] * 4 + mean_t * case["hq"] * case["d"] * 4) +
            b * case["k"] * 4, "flops": 4 * b * mean_t * case["hq"] * case["d"] * keys}


# ------------------------------------------------------------------ 64 bits
def _exact_norm_rope(st):
    c = st["case"]

    def rotated(y, table):
        n, h, d = y.shape
        half = table.shape[1] // 2
        ang = table[st["pos"].long()].double()
        z = torch.complex(ang[:, :half], ang[:, half:])[:, None, :]
        first = torch.arange(half, device="cuda") * (2 if c["inter"] else 1)
        second = first + (1 if c["inter"] else half)
        r = torch.complex(y[..., first], y[..., second]) * z
        y = y.clone()
        y[..., first], y[..., second] = r.real, r.imag
        return y

    def quantised(y):
        scale = y.abs().max(-1).values.clamp(min=1e-12) / 448
        return y / scale.unsqueeze(-1), scale

    q, k, qI, kI = (st[n].double() for n in ("q", "k", "qI", "kI"))
    q = q / (q.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * st["q_weight"].double()
    k = k / (k.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6).sqrt() * st["k_weight"].double()
    var, mean = torch.var_mean(kI, -1, correction=0, keepdim=True)
    kI = (kI - mean) / (var + 1e-6).sqrt() * st["kI_weight"].double() + st["kI_bias"].double()
    rows = torch.nonzero(st["slot"] >= 0)[:, 0]
    at = st["slot"][rows]
    K, V = st["K"].double(), st["V"].double()
    K[at], V[at] = rotated(k, st["rope"])[rows], st["v"].double()[rows]
    k8, ks = quantised(rotated(kI, st["ropeI"]))
    kI8 = torch.zeros(st["kI8"].shape, dtype=torch.float64, device="cuda")
    kI_scale = st["kI_scale"].double()
    kI8[at], kI_scale[at] = k8[rows], ks[rows]
    out = dict(Q=rotated(q, st["rope"]), K=K, V=V, kI8=kI8, kI_scale=kI_scale)
    if c["q8"]:
        out["qI8"], out["qI_scale"] = quantised(rotated(qI, st["ropeI"]))
    else:
        out["qI"] = rotated(qI, st["ropeI"])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(st)
    out = (st["scores"] if case["op"] == "tree_score" else st["out"]).double()
    prefix, draft, masks = st["prefix"].tolist(), st["draft"].tolist(), st["mask"].tolist()
    t = case["t"]
    for b in range(case["b"]):
        n, m = prefix[b], draft[b]
        tree = torch.tensor([[masks[b][i] >> u & 1 for u in range(m)] for i in range(m)],
                            dtype=torch.bool, device="cuda")
        if case["op"] == "tree_score":
            k8 = st["kI8"][b, :n + m].view(torch.float8_e4m3fn).double()
            k = k8 * st["kI_scale"][b, :n + m, None].double()
            for i in range(m):
                dots = torch.relu(st["q"][b, i].double() @ k.T)
                score = st["w"][b, i].double() @ dots
                score[n:][~tree[i]] = -math.inf
                out[b * t + i, :n + m] = score
            continue
        if st["idx"] is None:
            rows = torch.arange(n, device="cuda")
        else:
            rows = st["idx"][b][st["idx"][b] >= 0].long()
        rows = torch.cat([rows, n + torch.arange(m, device="cuda")])
        k, v = st["K"][b, rows].double(), st["V"][b, rows].double()
        z = torch.einsum("thd,sd->ths", st["Q"][b, :m].double(), k) / math.sqrt(case["d"])
        hidden = torch.zeros((m, rows.numel()), dtype=torch.bool, device="cuda")
        hidden[:, rows.numel() - m:] = ~tree
        z = z.masked_fill(hidden[:, None, :], -math.inf)
        out[b, :m] = torch.einsum("ths,sd->thd", torch.softmax(z, -1), v)
    return out
