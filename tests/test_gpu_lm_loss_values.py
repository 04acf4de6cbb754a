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
    logits = torch.tensor([[low, low, low], [low, 0.0, 1.0], [high, high, 0.0], [high, low, high],
                           [0.9 * high, high, 1.0], [-torch.inf, low, low]])
    if tau < 1.0:
        logits[1] *= torch.tensor([1.0, tau, tau])
    ids = torch.tensor([[5, 0, 299]] * 6, dtype=I32)
    Case(x, w, dloss, ids=ids, logits=logits, tau=tau).check()


# --------------------------------------------------------------- what the factor on the logits does

FACTOR = 2.0 ** -30  # per element of D, up to 65536 of them


def given_back(D):
    return min(D, 65536) * FACTOR


@pytest.mark.parametrize("D", [64, 1024, 4096, 65536, 1 << 20])
def test_rows_of_one_element_are_off_by_the_factor_at_most(D):
    # their products are exact and lose nothing, so the factor is all that they can be off by
    T, V = 16, 40
    x = torch.zeros(T, D)
    x[torch.arange(T), torch.randint(0, D, (T,), generator=gen(60))] = 20 * torch.randn(T, generator=gen(61))
    x, w, t = x.to(BF16), torch.randn(V, D, generator=gen(62)).to(BF16), torch.randint(0, V, (T,), generator=gen(63))
    loss, lse = ce_fwd(x, w, t)
    z = x.double() @ w.double().T
    want, zt = torch.logsumexp(z, 1), z.gather(1, t[:, None])[:, 0]
    size = z.abs().amax(1)
    bound = 1.01 * given_back(D) * size + R.U32 * (8 * (size + want.abs() + 2) + 64)
    R.check(lse, want, bound, "lse")
    R.check(loss, want - zt, 2 * bound, "loss")


@pytest.mark.parametrize("D", [1024, 4096, 16384])
def test_the_factor_gives_back_what_rows_that_lean_lose(D):
    # with one word, lse is its logit. On average no more than half of the factor is left, whichever way: without it
    # the mean is off by the whole of it
    T = 256
    w = (torch.randn(1, D, generator=gen(D + 64)) / D ** 0.5).to(BF16)
    x = (torch.randn(T, D, generator=gen(D + 65)) + 8 * w.float()).to(BF16)
    _, lse = ce_fwd(x, w, torch.zeros(T))
    z = (x.double() @ w.double().T)[:, 0]
    rows = z > 4
    assert rows.sum() > T // 2
    off = (lse.cpu().double() / z - 1)[rows].mean()
    assert abs(float(off)) < 0.5 * given_back(D), float(off) / given_back(D)


# ------------------------------------------------------------------- gradients against differences

@pytest.mark.parametrize("kind", ["ce", "distill"])
@pytest.mark.parametrize("of", ["w", "x"])
def test_the_softmax_part_of_the_gradient_is_the_difference_of_the_forward(kind, of):
    # Moved is what the targets' part of the gradient does not see: rows of w that are nobody's target, or columns
    # of x in which the targets' rows are 0. All terms have one sign, so nothing cancels.
    T, D, V, cols, h = 64, 64, 40, 8, 1.0 / 256
    x = torch.randint(0, 16, (T, D), generator=gen(70)).float() / 16
    w = torch.randint(-8, 9, (V, D), generator=gen(71)).float() / 16
    w[V // 2:, :cols] = torch.randint(4, 9, (V // 2, cols), generator=gen(72)).float() / 16
    w[:V // 2, :cols] = 0.0
    move = torch.zeros(V, D) if of == "w" else torch.zeros(T, D)
    move[V // 2 if of == "w" else 0:, :cols] = 1.0
    dloss = 0.5 + torch.rand(T, generator=gen(73))
    if kind == "ce":
        kw = dict(targets=torch.randint(0, V // 2, (T,), generator=gen(74)).to(I32))
    else:
        kw = dict(ids=torch.randint(0, V // 2, (T, 3), generator=gen(74)).to(I32),
                  logits=torch.randn(T, 3, generator=gen(75)), tau=2.0)

    def case(s):
        xs, ws = (x, w + s * h * move) if of == "w" else (x + s * h * move, w)
        assert torch.equal(xs.to(BF16).float(), xs) and torch.equal(ws.to(BF16).float(), ws)  # moved by exact steps
        return Case(xs.to(BF16), ws.to(BF16), dloss, **kw)

    up, down = (case(s).fwd()[0].double().cpu() for s in (1, -1))
    diff = float(((up - down) * dloss.double()).sum()) / (2 * h)
    c = case(0)
    dx, dw = c.bwd(c.fwd()[1])
    got = float(((dw if of == "w" else dx).double().cpu() * move.double()).sum())
    # dl and the result each rounded by half a bf16 step; a third derivative of at most a tenth of the cube of
    # what the logits move per unit; and the fp32 losses, a few steps of the logits' products, over 2 h
    tau = kw.get("tau", 1.0)
    a = float((x[:, :cols].sum(1) if of == "w" else w[V // 2:, :cols].sum(1)).max()) / tau
    size = float((x.double() @ w.double().abs().T).max()) / tau
    bound = 2 * 2.0 ** -8 * abs(got) + float(dloss.sum()) * tau * tau * (
        0.1 * a ** 3 * h * h / 6 + 2 * (20 * R.ACC * size + 64 * R.U32 * 8) / (2 * h))
    assert bound < 0.05 * abs(got), (bound, got)
    assert abs(diff - got) < bound, (diff, got, bound)


# ----------------------------------------------------------------------- weights past 32 bits, and pieces

def test_dx_from_weights_past_32_bits():
    # dx comes from rows of w on both sides of 2^31 elements, summed over slices of the vocabulary. An eighth of the
    # rows, one after another, has a value of its own in every eighth column: a slice that is missed, or read from
    # elsewhere, shows in those columns. The targets' rows have none, so that theirs does not hide it.
    T, D, V, parts, value = 3, 4096, 600_003, 8, 1.0 / 16
    w = torch.randn(V, D, device="cuda", dtype=BF16).mul_(0.5 / D ** 0.5)
    targets = torch.tensor([V - 1, 524_288, 7], dtype=I32, device="cuda")
    step = -(-V // parts)
    for b in range(parts):
        w[b * step:(b + 1) * step, b::parts] += value
    w[targets.long()] = 0
    x = torch.randn(T, D // parts, parts, generator=gen(80))
    x = (x - x.mean(1, keepdim=True)).view(T, D).to(BF16).cuda()  # so that every eighth has about the same probability
    dloss = torch.tensor([1.0, -0.5, 2.0], device="cuda")
    z = torch.cat([x.double() @ w[a:a + 50_000].double().T for a in range(0, V, 50_000)], 1)
    lse = torch.logsumexp(z, 1).float()
    ws = B.alloc_workspace(B.moe_lm_workspace_bytes(T, D, V))
    dx = torch.full_like(x, 3.0)
    B.moe_lm_ce_bwd(x, w, targets, lse, dloss, dx, None, ws)
    assert B.moe_get_status(ws) == 0
    size = x.double().norm(dim=1)[:, None] * 2.0  # no row of w is longer: 0.5 at random and 1/16 in 512 columns
    dz = (D // 16 + 16) * R.ACC * size
    dl = dloss.double()[:, None] * torch.exp(z - lse.double()[:, None])
    # what an eighth adds to its columns
    share = value * torch.stack([dl[:, b * step:(b + 1) * step].sum(1).abs() for b in range(parts)], 1)
    dl[range(T), targets.long()] -= dloss.double()
    bdl = dl.abs() * (dz + 8 * R.U32 * (z.abs() + lse.double().abs()[:, None] + 2)) * 1.01 + R.round_bound(dl, BF16)
    want, bound = (torch.zeros(T, D, dtype=torch.double, device="cuda") for _ in range(2))
    for a in range(0, V, 50_000):
        part, rows = slice(a, a + 50_000), w[a:a + 50_000].double()
        want += dl[:, part] @ rows
        bound += bdl[:, part] @ rows.abs() + (V // 16 + 64) * R.ACC * (dl[:, part].abs() @ rows.abs())
    bound = 1.01 * bound + R.round_bound(want, BF16)
    columns = torch.arange(D, device="cuda") % parts
    assert (bound < 0.5 * share[:, columns] / 8).all()  # half of what a slice of a sixty-fourth adds
    R.check(dx, want, bound, "dx")


def test_both_gradients_in_one_grid_over_several_pieces():
    # 2 T V bytes pass the 512 MB of a piece, with few enough rows and weights for the joint grid
    T, D, V = 512, 64, 600_001
    x, w, dloss = head(T, D, V, 81)
    t = torch.randint(0, V, (T,), generator=gen(82)).to(I32)
    t[::5] = -100
    t[1], t[2], t[3] = V - 1, V // 2, 300_032
    c = Case(x, w, dloss, targets=t)
    lse = c.fwd()[1]
    dx, dw = c.bwd(lse)
    assert B.moe_get_status(c.ws) == 0
    want = R.lm_bwd(c.dev["x"], c.dev["w"], c.sparse("cuda"), lse, c.dev["dloss"], 1.0)
    R.check(dx, want[0], want[2], "dx")
    R.check(dw, want[1], want[3], "dw")
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), c.bwd(lse)))
