"""Values of the vocabulary losses where a bound of the logits' size would hide an error: rows that are sure of
their target, what the factor on the logits does, teacher logits at the ends of their type, and weights past 32
bits. Against 64-bit values, within bounds that follow the loss itself."""

import pytest
import torch

import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B
from test_gpu_lm_loss import Case, head

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ce_fwd(x, w, targets):
    T, D, V = *x.shape, w.shape[0]
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    ws = B.alloc_workspace(B.moe_lm_workspace_bytes(T, D, V))
    B.moe_lm_ce_fwd(x.cuda(), w.cuda(), targets.to(I32).cuda(), loss, lse, ws)
    assert B.moe_get_status(ws) == 0
    return loss, lse


def distill_fwd(x, w, ids, logits, tau):
    T, D, V = *x.shape, w.shape[0]
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    ws = B.alloc_workspace(B.moe_lm_workspace_bytes(T, D, V, ids.shape[1]))
    B.moe_lm_distill_fwd(x.cuda(), w.cuda(), ids.to(I32).cuda(), logits.cuda(), loss, lse, ws, tau)
    assert B.moe_get_status(ws) == 0
    return loss, lse


# --------------------------------------------------------------------------- rows sure of their target

def sure_rows(D, lo, hi, T=300, V=2000):
    """Rows whose target's logit lies about lo to hi above the others'."""
    w = (torch.randn(V, D, generator=gen(D)) / D ** 0.5).to(BF16)
    t = torch.randint(0, V, (T,), generator=gen(D + 1))
    lean = lo + (hi - lo) * torch.rand(T, 1, generator=gen(D + 2))
    return (0.3 * torch.randn(T, D, generator=gen(D + 3)) + lean * w[t].float()).to(BF16), w, t


def sure_loss(x, w, t, tau=1.0):
    """-log q of the target at the temperature, and its bound: the other terms' relative errors (both logits', with
    what is given back of them, and the exponent's rounding), and the sum's additions, each half a step of 1."""
    z, dz = R._z(x, w, tau)
    zt = z.gather(1, t[:, None])
    rest = torch.exp(z - zt).scatter(1, t[:, None], 0.0)
    rel = 2.5 * dz.amax(1, keepdim=True) + 4 * R.U32 * (z - zt).abs() + 8 * R.U32
    loss = torch.log1p(rest.sum(1))
    assert (zt >= z).all()
    return loss, (rest * rel).sum(1) * 1.01 + (48 + w.shape[0] // 512) * R.U32


@pytest.mark.parametrize("lo,hi", [(8, 20), (30, 64), (200, 400)])
@pytest.mark.parametrize("D", [64, 832, 2048, 4096, 7168])
def test_cross_entropy_of_rows_that_are_sure(D, lo, hi):
    x, w, t = sure_rows(D, lo, hi)
    if D == 64 or lo == 8:  # keep the rows whose target is the largest logit
        keep = (x.double() @ w.double().T).argmax(1) == t
        x, t = x[keep], t[keep]
    loss, _ = ce_fwd(x, w, t)
    R.check(loss, *sure_loss(x, w, t), "loss")
    assert (loss >= 0).all()


@pytest.mark.parametrize("tau", [0.5, 2.0])
@pytest.mark.parametrize("D", [832, 4096])
def test_distillation_of_rows_that_are_sure(D, tau):
    x, w, t = sure_rows(D, 30, 200)
    want, bound = sure_loss(x, w, t, tau)
    ids = torch.full((x.shape[0], 3), -1)
    ids[:, 1] = t
    one = distill_fwd(x, w, ids, torch.randn(ids.shape, generator=gen(5)), tau)[0]  # one kept entry: p = 1
    logits = torch.full(ids.shape, -1e9)
    logits[:, 1] = 4.0
    ids[:, 0], ids[:, 2] = (t + 1) % w.shape[0], (t + 2) % w.shape[0]
    far = distill_fwd(x, w, ids, logits, tau)[0]  # the others' p is 0
    for loss in (one, far):
        R.check(loss, tau * tau * want, tau * tau * (bound + 4 * R.U32 * want), "loss")
        assert (loss >= 0).all()


# ------------------------------------------------------------- teacher logits at the ends of their type

@pytest.mark.parametrize("tau", [2.0 ** -10, 0.5, 0.9, 1.0, 4.0])
def test_teacher_logits_at_the_ends_of_their_type(tau):
    x, w, dloss = head(6, 64, 300, 50)
    x = (x.float() * min(1.0, tau)).to(BF16)  # the student's logits stay ordinary at the temperature
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    logits = torch.tensor([[low, low, low], [low, 0.0, 1.0], [high, high, 0.0], [high, low, high], [0.9 * high, high, 1.0],
                           [-torch.inf, low, low]])
    if tau < 1.0:
        logits[1] *= torch.tensor([1.0, tau, tau])
    ids = torch.tensor([[5, 0, 299]] * 6, dtype=I32)
    Case(x, w, dloss, ids=ids, logits=logits, tau=tau).check()
