"""64-bit values of the operators around the expert layer, from their definitions, and the error
bounds the kernels are held to. No package code here."""

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
ACC = 2.0 ** -23  # one truncated fp32 addition, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def round_bound(ref, dtype):
    """Rounding a value near ref to dtype: half a step, or half the smallest subnormal."""
    fi = torch.finfo(dtype)
    return ref.abs() * half_step(dtype) + fi.tiny * fi.eps / 2


def check(got, ref, bound, what=""):
    got = got.detach().double().cpu()
    ref, bound = ref.cpu(), bound.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{float(got[i])} against {float(ref[i])}, bound {float(bound[i])}")


# ------------------------------------------------------------------------------------ layer norm

def ln_fwd(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + eps).rsqrt()
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def ln_fwd_bounds(x, gamma, beta, eps, dtype):
    """A thread adds at most 32 values (or D / 512 of a long row), then 5 + 16 partial sums meet: the sums
    are off by at most n steps of the mean magnitude, and everything after by a few steps."""
    y, mean, rstd = ln_fwd(x, gamma, beta, eps)
    n = 32 + x.shape[1] // 512 + 24
    mag = x.double().abs().mean(1)
    dm = n * U32 * mag
    drel = 2 * n * U32 + (dm * rstd).square() + 8 * U32
    xhat = (x.double() - mean[:, None]).abs() * rstd[:, None]
    g = torch.ones_like(xhat) if gamma is None else gamma.double().abs()
    b = torch.zeros_like(xhat) if beta is None else beta.double().abs()
    dy = (dm * rstd)[:, None] * g + xhat * g * (drel[:, None] + 4 * U32) + 2 * U32 * (xhat * g + b)
    return dy * 1.01 + round_bound(y, dtype), dm + 2 * U32 * mean.abs(), drel * rstd


def ln_bwd(dy, x, gamma, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    g = dy if gamma is None else dy * gamma.double()
    xhat = (x - mean) * rstd
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def ln_bwd_bounds(dy, x, gamma, mean, rstd, dtype, param_dtype):
    dx, dgamma, dbeta = ln_bwd(dy, x, gamma, mean, rstd)
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    T, D = x.shape
    g = (dy if gamma is None else dy * gamma.double()).abs()
    xhat = ((x - mean) * rstd).abs()
    n = 32 + D // 512 + 24 + 8  # the row sums, as in the forward, and the products' own roundings
    bdx = n * U32 * rstd * (g + g.mean(1, keepdim=True) + 2 * xhat * (g * xhat).mean(1, keepdim=True))
    k = min(T, T // 64 + 400) + 8  # a column's sum: a block's rows one after another, then the blocks
    bdg = k * U32 * (dy.abs() * xhat).sum(0)
    bdb = k * U32 * dy.abs().sum(0)
    return (bdx + round_bound(dx, dtype), bdg + round_bound(dgamma, param_dtype),
            bdb + round_bound(dbeta, param_dtype))


# ---------------------------------------------------------------------------------------- router

def router_fwd(logits, K, normalize):
    z = logits.double()
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    scores = torch.softmax(top, 1) if normalize else torch.softmax(z, 1).gather(1, ids)
    dead = torch.isneginf(z).all(1, keepdim=True)
    return ids, torch.where(dead, 0.0, scores)


def router_bwd(logits, ids, ds, normalize):
    z, ds, ids = logits.double(), ds.double(), ids.long()
    mask = torch.zeros_like(z, dtype=torch.bool).scatter(1, ids, True)
    base = torch.where(mask, z, -torch.inf) if normalize else z
    p = torch.softmax(base, 1)
    dead = torch.isneginf(base).all(1, keepdim=True)
    p = torch.where(dead, 0.0, p)
    full = torch.zeros_like(z).scatter(1, ids, ds)
    dot = (p * full).sum(1, keepdim=True)
    # the same shape of magnitudes bounds the error
    return p * (full - dot), p * (full.abs() + 2 * (p * full.abs()).sum(1, keepdim=True))


def router_rel(logits):
    """Relative error of a score: the exponents' rounding, exp's two units, and sums of up to 48 terms one
    after another (32 of a lane, then the warp and the block)."""
    z = logits.double()
    z = torch.where(torch.isfinite(z) & (z > -1e30), z, 0.0)
    spread = float((z.amax(1) - z.amin(1)).max())
    return (4 * (spread + 4) + 64) * U32


# ------------------------------------------------------------------------------- vocabulary losses

def teacher(ids, logits, tau):
    """p, p log p summed, and the rows that have a distribution."""
    kept = ids >= 0
    a = torch.where(kept, logits.double() / tau, -torch.inf)
    has = (kept & ~torch.isneginf(a)).any(1)
    p = torch.where(has[:, None], torch.softmax(a, 1), 0.0)
    return p, torch.special.xlogy(p, p).sum(1), has


def _z(x, w, tau):
    """Scaled logits, and how far the tensor cores' fp32 sums of D products may be from them."""
    x, w = x.double(), w.double()
    n = x.shape[1] // 16 + 16
    return (x @ w.T) / tau, n * ACC * (x.abs() @ w.abs().T) / tau


def sparse(targets=None, ignore=-100, teacher_ids=None, teacher_logits=None, tau=1.0):
    """Both losses as (ids [T,K], p [T,K], sum p log p, rows that count)."""
    if targets is not None:
        has = (targets != ignore) & (targets >= 0)
        return targets.long()[:, None], has.double()[:, None], torch.zeros_like(targets, dtype=torch.double), has
    p, ent, has = teacher(teacher_ids, teacher_logits, tau)
    return teacher_ids.long(), p, ent, has


def lm_fwd(x, w, target, tau):
    """loss, lse and their bounds."""
    ids, p, ent, has = target
    z, dz = _z(x, w, tau)
    V = z.shape[1]
    lse = torch.logsumexp(z, 1)
    at = ids.clamp(0, V - 1)
    zt, dzt = z.gather(1, at), dz.gather(1, at)
    loss = torch.where(has, tau * tau * (ent + (p * (lse[:, None] - zt)).sum(1)), 0.0)
    # lse: the logits' error, exponents rounded at magnitude |z| + |lse|, a sum of 256 terms per tile and the tiles'
    blse = dz.amax(1) + 8 * U32 * (z.abs().amax(1) + lse.abs() + 2) + (300 + V // 4096) * U32
    n = ids.shape[1] + 8
    pe = 64 * U32 * (1 + (torch.special.xlogy(p, p).abs().sum(1)))  # the teacher's own softmax
    bloss = tau * tau * (blse + (p * dzt).sum(1) + n * U32 * (p * (lse[:, None] - zt).abs()).sum(1)
                         + n * U32 * (lse.abs() + ent.abs()) + pe * (1 + (lse[:, None] - zt).abs().amax(1)))
    return loss, lse, torch.where(has, bloss, 0.0), blse


def lm_bwd(x, w, target, lse, dloss, tau):
    """dx, dw and their bounds, for the given lse (rounded as the caller's is)."""
    ids, p, _, has = target
    z, dz = _z(x, w, tau)
    T, V = z.shape
    q = torch.exp(z - lse.double()[:, None])
    c = torch.where(has, tau * dloss.double(), 0.0)[:, None]
    hot = torch.zeros_like(z).scatter_add(1, ids.clamp(0, V - 1), p)
    dl = c * (q - hot)
    # dl: the exponent's error, the teacher's, one bf16 rounding
    e = dz + 8 * U32 * (z.abs() + lse.double().abs()[:, None] + 2)
    bdl = c.abs() * (q * e * 1.01 + 128 * U32 * hot + 4 * U32 * (q + hot)) + round_bound(dl, torch.bfloat16)
    xd, wd = x.double(), w.double()
    dx, dw = dl @ wd, dl.T @ xd
    bdx = bdl @ wd.abs() + (V // 16 + 64) * ACC * (dl.abs() @ wd.abs())
    bdw = bdl.T @ xd.abs() + (T // 16 + 64) * ACC * (dl.abs().T @ xd.abs())
    return dx, dw, bdx * 1.01 + round_bound(dx, torch.bfloat16), bdw * 1.01 + round_bound(dw, torch.bfloat16)
