"""Plain 64-bit forms of the drafted-token operators, with error bounds.

Written from the formulas in include/indexcache.h with torch double tensors
on the CPU (no code of the library).  Each returns the result and, beside
it, how far a kernel may be off, counted from its roundings:
  u32 = 2^-24 per fp32 operation (2^-23 where the tensor core may truncate),
  2^-8 for a bf16 rounding, 2^-4 (or half the smallest step) for e4m3."""
import math

import torch

U32, U32T, UBF16, UE4M3 = 2.0 ** -24, 2.0 ** -23, 2.0 ** -8, 2.0 ** -4


def visible(prefix, draft, mask, T):
    """[T, m] bool: which of the m drafts each row sees (mask None: a chain)."""
    see = torch.zeros((T, draft), dtype=torch.bool)
    for t in range(T):
        for u in range(draft):
            see[t, u] = u <= t if mask is None else bool(int(mask[t]) >> u & 1)
    return see


def tree_scores(q, w, k8, scale, prefix, draft, mask):
    """One sequence: q [T, H, d], w [T, H], k8 uint8 [S, d], scale [S].  Returns (scores, tol)
    [draft, prefix + draft] of the live rows."""
    n = prefix + draft
    k = k8[:n].view(torch.float8_e4m3fn).double()
    q, w, sc = q[:draft].double(), w[:draft].double(), scale[:n].double()
    H, d = q.shape[1], q.shape[2]
    dots = torch.einsum("thd,sd->ths", q, k)
    mags = torch.einsum("thd,sd->ths", q.abs(), k.abs())
    relu = dots.clamp_min(0)
    s = torch.einsum("th,ths->ts", w, relu) * sc
    # d products summed in fp32, then H weighted terms, the scale and the store
    tol = (torch.einsum("th,ths->ts", w.abs(), mags) * d +
           torch.einsum("th,ths->ts", w.abs(), relu) * (H + 3)) * sc * U32T
    see = visible(prefix, draft, mask, draft)
    s[:, prefix:][~see] = -math.inf
    return s, tol


def tree_attn(Q, K, V, prefix, draft, mask, idx, scale):
    """One sequence: Q [T, Hq, d], K, V [S, d], idx [k] or None.  Returns (out, tol) [draft, Hq, d]."""
    rows = torch.arange(prefix) if idx is None else idx[idx >= 0].long()
    rows = torch.cat([rows, prefix + torch.arange(draft)])
    see = torch.cat([torch.ones((draft, rows.numel() - draft), dtype=torch.bool),
                     visible(prefix, draft, mask, draft)], 1)
    # a slot that no row sees takes no part, whatever it holds
    used = see.any(0)
    rows, see = rows[used], see[:, used]
    q, k, v = Q[:draft].double(), K[rows].double(), V[rows].double()
    d = q.shape[2]
    if rows.numel() == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    z = torch.einsum("thd,sd->ths", q, k) * scale
    zmag = torch.einsum("thd,sd->ths", q.abs(), k.abs()) * scale
    z = z.masked_fill(~see[:, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l.clamp_min(1e-300), torch.zeros_like(p))
    out = torch.einsum("ths,sd->thd", p, v)
    mean_abs = torch.einsum("ths,sd->thd", p, v.abs())
    # logits: d products and the scale in fp32; a weight is off by twice the
    # largest logit error, by its own rounding to bf16, and by exp2's 2^-22;
    # two sums of all weights in fp32; one rounding of the output
    dz = (zmag * see[:, None, :]).amax(-1, keepdim=True) * (d + 4) * U32T
    tol = out.abs() * UBF16 + mean_abs * (UBF16 * 1.01 + 2 * dz + 2.0 ** -21 +
                                          2 * rows.numel() * U32T) + 1e-30
    return out, tol


def norm_rope(x, norm, weight, bias, eps, rope, pos, interleaved):
    """x [rows, H, d]; returns (z, tol before the output's rounding)."""
    x = x.double()
    d = x.shape[-1]
    r = torch.ones_like(x[..., :1])
    tol = torch.zeros_like(x)
    y = x
    wt = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    if norm is not None:
        mu = x.mean(-1, keepdim=True) if norm == "layer" else 0.0 * r
        y = x - mu
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        shift = x.abs().mean(-1, keepdim=True) * (d + 2) * U32 if norm == "layer" else 0.0 * r
        y = y * r * wt
        # the mean's error moves each value and, to first order, not the deviation
        tol = shift * r * wt.abs() * 2 + y.abs() * (d / 2 + 8) * U32
        if bias is not None:
            y = y + bias.double()
            tol = tol + y.abs() * U32
    if rope is None:
        return y, tol
    dr = rope.shape[1]
    cs = rope[pos.long()].double()[:, None, :]
    c, s = cs[..., :dr // 2], cs[..., dr // 2:]
    ia = torch.arange(dr // 2) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else dr // 2)
    a, b = y[..., ia], y[..., ib]
    ta, tb = tol[..., ia], tol[..., ib]
    z, tz = y.clone(), tol.clone()
    z[..., ia], z[..., ib] = a * c - b * s, b * c + a * s
    more = (a.abs() + b.abs()) * 3 * U32
    tz[..., ia] = ta * c.abs() + tb * s.abs() + more
    tz[..., ib] = tb * c.abs() + ta * s.abs() + more
    return z, tz
