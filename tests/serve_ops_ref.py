"""64-bit values of the operators of a decoding step, from their definitions, and the error bounds the kernels
are held to. No package code here. Runs on the tensors' device."""

import torch

import train_ops_ref as R
from train_ops_ref import ACC, U32, half_step, round_bound

BF16 = torch.bfloat16


# ------------------------------------------------------------------------ the layer for a few tokens

def few(x, ids, scores, w13, w2):
    """out and its bound. Pairs with a score of 0 or an id outside [0, E) contribute nothing, whatever the
    weights hold.

    The bound: an fp32 sum of n products in steps of 16, each cut off, and then 8 warps' sums; H's rounding
    to bf16; the exponential (2 + 1.2 |g| units); the pairs one after another."""
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
        dh = dh * 1.01 + round_bound(h, BF16)
        y = h @ wd.T
        dy = dh @ wd.abs().T + (F // 16 + 16) * ACC * (h.abs() @ wd.abs().T)
        out.index_add_(0, t, s * y)
        err.index_add_(0, t, s.abs() * dy)
        mag.index_add_(0, t, s.abs() * (h.abs() @ wd.abs().T))
    err = err + (ids.shape[1] + 10) * U32 * mag
    return out, err * 1.01 + round_bound(out, BF16)
