"""64-bit values of the norms around a block, forward and backward, from their definitions, and the error bounds
the kernels are held to. No package code here."""

import torch

from train_ops_ref import U32, round_bound


def _d(t):
    return None if t is None else t.double()


def _steps(D):
    """Additions that a row's sum takes one after another: a thread's own, its group's, and the products' roundings."""
    return 32 + D // 512 + 24


def fwd(block, residual, post_gamma, gate, pre_gamma, scale, eps, post):
    """stream, normed, post_rstd (None without a norm after the block), pre_rstd; and u."""
    u, post_rstd = _d(block), None
    if post:
        post_rstd = (u.square().mean(1) + eps).rsqrt()
        u = u * post_rstd[:, None]
        u = u if post_gamma is None else u * _d(post_gamma)
    u = u if gate is None else u * _d(gate)
    a = scale * _d(residual) + u
    pre_rstd = (a.square().mean(1) + eps).rsqrt()
    normed = a * pre_rstd[:, None]
    return a, normed if pre_gamma is None else normed * _d(pre_gamma), post_rstd, pre_rstd, u


def fwd_bounds(block, residual, post_gamma, gate, pre_gamma, scale, eps, post, dtype):
    """A sum of n squares is off by n steps of itself at most, and what comes after by a few."""
    a, normed, post_rstd, pre_rstd, u = fwd(block, residual, post_gamma, gate, pre_gamma, scale, eps, post)
    n = _steps(a.shape[1]) * U32
    da = (n + 6 * U32) * u.abs() + 2 * U32 * ((scale * _d(residual)).abs() + u.abs())
    rel = da.square().mean(1).sqrt() * pre_rstd + n + 6 * U32
    g = 1.0 if pre_gamma is None else _d(pre_gamma).abs()
    dn = da * pre_rstd[:, None] * g + normed.abs() * (rel[:, None] + 4 * U32)
    return (da * 1.01 + round_bound(a, dtype), dn * 1.01 + round_bound(normed, dtype),
            (n + 6 * U32) * post_rstd if post else None, rel * 1.01 * pre_rstd)


def bwd(dstream, dnormed, block, stream, post_gamma, gate, pre_gamma, post_rstd, pre_rstd, scale):
    """(dblock, dresidual, dpost_gamma, dgate, dpre_gamma) and their bounds before the last rounding. The gradients of
    a [T,D] gate have its shape; those of what is not there are None."""
    dn, st = _d(dnormed), _d(stream)
    T, D = st.shape
    n = (_steps(D) + 8) * U32
    k = (min(T, T // 64 + 400) + 8) * U32  # a column's sum: a block's rows one after another, then the blocks
    pre = _d(pre_rstd)[:, None]
    hat = st * pre
    gn = dn if pre_gamma is None else dn * _d(pre_gamma)
    m1 = (gn * hat).mean(1, keepdim=True)
    ds = torch.zeros_like(st) if dstream is None else _d(dstream)
    da = ds + pre * (gn - hat * m1)
    eda = pre * (hat.abs() * n * (gn * hat).abs().mean(1, keepdim=True) + 6 * U32 * (gn.abs() + (hat * m1).abs()))
    eda = eda + 2 * U32 * (ds.abs() + da.abs())
    dpre, edpre = (dn * hat).sum(0), k * (dn * hat).abs().sum(0)
    res, eres = scale * da, abs(scale) * eda + 2 * U32 * (scale * da).abs()
    post = None if post_rstd is None else _d(post_rstd)[:, None]
    bh = torch.zeros_like(st) if block is None else _d(block) * (1.0 if post is None else post)
    w = 1.0 if post_gamma is None else _d(post_gamma)
    g = 1.0 if gate is None else _d(gate)
    gb, egb = da * g * w, (eda + 4 * U32 * da.abs()) * abs(g * w)
    db, edb = gb, egb + 2 * U32 * gb.abs()
    if post is not None:
        m2 = (gb * bh).mean(1, keepdim=True)
        em2 = (egb * bh.abs()).mean(1, keepdim=True) + n * (gb * bh).abs().mean(1, keepdim=True)
        db = post * (gb - bh * m2)
        edb = post * (egb + bh.abs() * em2 + 6 * U32 * (gb.abs() + (bh * m2).abs()))
    dpost = edpost = dgate = edgate = None
    each, eeach = da * bh, eda * bh.abs() + 4 * U32 * (da * bh).abs()
    if gate is not None and gate.dim() == 2:
        dgate, edgate = each * w, eeach * abs(w) + 4 * U32 * (each * w).abs()
        if post is not None:
            dpost, edpost = (each * g).sum(0), (eeach * g.abs()).sum(0) + k * (each * g).abs().sum(0)
    else:
        s, es = each.sum(0), eeach.sum(0) + k * each.abs().sum(0)
        if gate is not None:
            dgate, edgate = s * w, (es + 2 * U32 * s.abs()) * abs(w)
        if post is not None:
            dpost, edpost = s * g, (es + 2 * U32 * s.abs()) * abs(g)
    return (db, res, dpost, dgate, dpre), tuple(None if e is None else e * 1.01 for e in (edb, eres, edpost, edgate, edpre))
