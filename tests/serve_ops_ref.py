"""64-bit values of the operators of a decoding step, from their definitions, and the error bounds the kernels
are held to. No package code here. Runs on the tensors' device."""

import math

import torch

from train_ops_ref import ACC, U32, half_step, round_bound

BF16 = torch.bfloat16


# ------------------------------------------------------------------------ the layer for a few tokens

def few(x, ids, scores, w13, w2):
    """out and its bound. Pairs with a score of 0 or an id outside [0, E) contribute nothing, whatever the
    weights hold.

    The bound: an fp32 sum of n products in steps of 16, each cut off, and then 8 warps' sums; H's rounding
    to two bf16 parts; the exponential (2 + 1.2 |g| units); the pairs one after another."""
    T, D = x.shape
    E, _, F, _ = w13.shape
    out = torch.zeros(T, D, dtype=torch.double, device=x.device)
    err = torch.zeros_like(out)
    mag = torch.zeros_like(out)
    ok = (ids >= 0) & (ids < E) & (scores != 0)
    for e in torch.unique(ids[ok]).tolist():
        t, k = torch.nonzero((ids == e) & ok, as_tuple=True)
        s = scores[t, k].double()[:, None]
        xe, wg, wu, wd = x[t].double(), w13[e, 0].double(), w13[e, 1].double(), w2[e].double()
        g, u = xe @ wg.T, xe @ wu.T
        n = D // 16 + 16
        dg, du = n * ACC * (xe.abs() @ wg.abs().T), n * ACC * (xe.abs() @ wu.abs().T)
        silu = g / (1 + torch.exp(-g))
        h = silu * u
        dh = 1.11 * dg * (u.abs() + du) + silu.abs() * du + (6 + 2 * g.abs()) * ACC * h.abs()
        dh = dh * 1.01 + h.abs() * half_step(BF16) ** 2 + 2.0 ** -130
        y = h @ wd.T
        dy = dh @ wd.abs().T + 2 * (F // 16 + 16) * ACC * (h.abs() @ wd.abs().T)
        out.index_add_(0, t, s * y)
        err.index_add_(0, t, s.abs() * dy)
        mag.index_add_(0, t, s.abs() * (h.abs() @ wd.abs().T))
    err = err + (ids.shape[1] + 10) * U32 * mag
    return out, err * 1.01 + round_bound(out, BF16)


# ------------------------------------------------------------------------ the choice of the next token

def sample_row(z, u, tau=1.0, k=0, p=1.0, least=0.0):
    """(token, log of its probability, distance to the nearest border) of one row in 64 bits, step by step. The distance
    says how far the choice is from another one, as a share of the weights: of the number to the borders of its token,
    and of the cut by share to the next tokens' running sums."""
    z = z.double()
    V = z.numel()
    if torch.isnan(z).any() or bool((z == -math.inf).all()):
        return -1, math.nan, math.inf
    order = torch.sort(z, descending=True, stable=True)[1]
    if not tau > 2.0 ** -60:
        return int(order[0]), 0.0, math.inf
    top = z[order[0]]
    w = torch.where(z == top, 1.0, torch.exp((z - top) / tau))
    w = torch.where(z == -math.inf, 0.0, w)
    kept, near = order, math.inf
    if 0 < k < V:
        kept = kept[:k]
    if p < 1.0:
        run = w[kept].cumsum(0) / w[kept].sum()
        n = int((run < p).sum()) + 1 if p > 0 else 1
        near = float((run[max(0, n - 2):n + 1] - p).abs().min()) if p > 0 else math.inf
        kept = kept[:n]
    if least > 0:
        kept = kept[w[kept] >= min(least, 1.0)]
    kept = torch.sort(kept)[0]
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24) if u == u else 0.0
    run = w[kept].cumsum(0)
    at = min(int((run <= u * run[-1]).sum()), kept.numel() - 1)
    share = run / run[-1]
    if u > 0:
        near = min(near, float((share - u).abs().min()))
    return int(kept[at]), math.log(float(w[kept[at]] / run[-1])), near
