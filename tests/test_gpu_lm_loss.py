"""The vocabulary losses on the GPU against their 64-bit values, within bounds counted from the bf16
roundings and the fp32 sums: ragged rows and vocabularies, ignored and empty rows, targets on tile
edges, several pieces of the vocabulary, absent gradients, other streams, graphs."""

import pytest
import torch

import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def head(T, D, V, seed):
    x = torch.randn(T, D, generator=gen(seed)).to(BF16)
    w = (2.0 * torch.randn(V, D, generator=gen(seed + 1)) / D ** 0.5).to(BF16)
    dloss = torch.randn(T, generator=gen(seed + 2))
    return x, w, dloss


class Case:
    """One problem: x, w and its targets, through the binding and through the reference."""

    def __init__(self, x, w, dloss, targets=None, ignore=-100, ids=None, logits=None, tau=1.0):
        self.x, self.w, self.dloss, self.tau, self.ignore = x, w, dloss, tau, ignore
        self.targets, self.ids, self.logits = targets, ids, logits
        self.dev = {k: v.cuda() for k, v in vars(self).items() if isinstance(v, torch.Tensor)}
        K = 1 if ids is None else ids.shape[1]
        self.T, self.D, self.V = x.shape[0], x.shape[1], w.shape[0]
        self.ws = B.alloc_workspace(B.moe_lm_workspace_bytes(self.T, self.D, self.V, K))
        self.ws.fill_(0xEE)  # what a workspace holds before a call must not matter

    def sparse(self, device="cpu"):
        if self.targets is not None:
            return R.sparse(targets=self.targets.to(device), ignore=self.ignore)
        return R.sparse(teacher_ids=self.ids.to(device), teacher_logits=self.logits.to(device), tau=self.tau)

    def fwd(self, stream=None):
        d = self.dev
        loss, lse = torch.full((self.T,), 7.0, device="cuda"), torch.full((self.T,), 7.0, device="cuda")
        if self.targets is not None:
            B.moe_lm_ce_fwd(d["x"], d["w"], d["targets"], loss, lse, self.ws, self.ignore, stream=stream)
        else:
            B.moe_lm_distill_fwd(d["x"], d["w"], d["ids"], d["logits"], loss, lse, self.ws, self.tau, stream=stream)
        return loss, lse

    def bwd(self, lse, dx=True, dw=True, stream=None):
        d = self.dev
        dx = torch.full_like(d["x"], 3.0) if dx else None
        dw = torch.full_like(d["w"], 3.0) if dw else None
        if self.targets is not None:
            B.moe_lm_ce_bwd(d["x"], d["w"], d["targets"], lse, d["dloss"], dx, dw, self.ws, self.ignore, stream=stream)
        else:
            B.moe_lm_distill_bwd(d["x"], d["w"], d["ids"], d["logits"], lse, d["dloss"], dx, dw, self.ws, self.tau,
                                 stream=stream)
        return dx, dw

    def check(self, status=0):
        loss, lse = self.fwd()
        assert B.moe_get_status(self.ws) == status
        want = R.lm_fwd(self.x, self.w, self.sparse(), self.tau)
        R.check(lse, want[1], want[3], "lse")
        R.check(loss, want[0], want[2], "loss")
        lse32 = want[1].float()
        dx, dw = self.bwd(lse32.cuda())
        assert B.moe_get_status(self.ws) == status
        rdx, rdw, bdx, bdw = R.lm_bwd(self.x, self.w, self.sparse(), lse32, self.dloss, self.tau)
        R.check(dx, rdx, bdx, "dx")
        R.check(dw, rdw, bdw, "dw")
        return loss, lse, dx, dw


def ce(T, D, V, seed=0, ignored=0.2):
    x, w, dloss = head(T, D, V, seed)
    t = torch.randint(0, V, (T,), generator=gen(seed + 3)).to(I32)
    t[torch.rand(T, generator=gen(seed + 4)) < ignored] = -100
    return Case(x, w, dloss, targets=t)


def distill(T, D, V, K, seed=0, tau=1.0):
    x, w, dloss = head(T, D, V, seed)
    ids = torch.randint(0, V, (T, K), generator=gen(seed + 3)).to(I32)  # some ids repeat within a row
    logits = 3.0 * torch.randn(T, K, generator=gen(seed + 4))
    gone = torch.rand(T, K, generator=gen(seed + 5)) < 0.2
    if T > 2:
        gone[1] = True  # nothing kept
    ids[gone] = -1
    return Case(x, w, dloss, ids=ids, logits=logits, tau=tau)


SIZES = [(1, 64, 1), (1, 64, 7), (5, 64, 255), (128, 128, 256), (129, 192, 257), (127, 64, 513), (300, 256, 1001),
         (17, 512, 3001), (64, 320, 640), (260, 1024, 300)]


@pytest.mark.parametrize("T,D,V", SIZES)
def test_cross_entropy(T, D, V):
    ce(T, D, V, seed=T + D + V).check()


@pytest.mark.parametrize("T,D,V,K,tau", [(1, 64, 1, 1, 1.0), (1, 64, 7, 3, 2.0), (5, 64, 255, 32, 0.5),
                                         (128, 128, 256, 33, 1.0), (129, 192, 257, 8, 4.0), (300, 256, 1001, 64, 2.0),
                                         (17, 512, 3001, 256, 1.0), (40, 64, 90, 100, 3.0)])
def test_distillation(T, D, V, K, tau):
    distill(T, D, V, K, seed=T + D + V + K, tau=tau).check()


def test_targets_on_the_edges_of_tiles_and_chunks():
    V = 1000
    edges = [0, 1, 30, 31, 32, 33, 63, 64, 255, 256, 257, 511, 512, 767, 768, 991, 992, 993, 998, 999]
    x, w, dloss = head(len(edges), 64, V, 5)
    Case(x, w, dloss, targets=torch.tensor(edges, dtype=I32)).check()
    ids = torch.tensor([edges, edges[::-1], [999] * 20, [31] * 10 + [32] * 10], dtype=I32)
    Case(x[:4], w, dloss[:4], ids=ids, logits=torch.randn(4, 20, generator=gen(6)), tau=1.5).check()


def test_all_rows_ignored():
    c = ce(140, 64, 300, seed=7, ignored=2.0)
    loss, _, dx, dw = c.check()
    assert not loss.any() and not dx.any() and not dw.any()


def test_an_ignore_index_inside_the_vocabulary():
    x, w, dloss = head(20, 64, 40, 8)
    t = torch.randint(0, 4, (20,), generator=gen(9)).to(I32)
    Case(x, w, dloss, targets=t, ignore=0).check()


def test_targets_outside_the_vocabulary_raise_the_status_bit():
    x, w, dloss = head(6, 64, 40, 10)
    bad = Case(x, w, dloss, targets=torch.tensor([3, 40, -5, 39, -100, 1 << 30], dtype=I32))
    good = Case(x, w, dloss, targets=torch.tensor([3, -100, -100, 39, -100, -100], dtype=I32))
    (loss, lse), (want, _) = bad.fwd(), good.fwd()
    assert B.moe_get_status(bad.ws) == B.MOE_DEV_BAD_TARGET and B.moe_get_status(good.ws) == 0
    assert torch.equal(loss, want)
    got, ref = bad.bwd(lse), good.bwd(lse)
    assert B.moe_get_status(bad.ws) == B.MOE_DEV_BAD_TARGET
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ids = torch.tensor([[3, 40, 5]] * 6, dtype=I32)
    logits = torch.randn(6, 3, generator=gen(11))
    bad = Case(x, w, dloss, ids=ids, logits=logits)
    good = Case(x, w, dloss, ids=torch.where(ids == 40, -1, ids), logits=logits)
    assert torch.equal(bad.fwd()[0], good.fwd()[0])
    assert B.moe_get_status(bad.ws) == B.MOE_DEV_BAD_TARGET and B.moe_get_status(good.ws) == 0


def test_what_stands_in_masked_teacher_entries_does_not_matter():
    x, w, dloss = head(7, 64, 300, 12)
    ids = torch.randint(0, 300, (7, 5), generator=gen(13)).to(I32)
    logits = torch.randn(7, 5, generator=gen(14))
    ids[:, 2] = -1
    ids[3] = -1
    want = None
    for junk in (0.0, float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min, 1e30):
        logits[:, 2] = junk
        logits[3] = junk
        c = Case(x, w, dloss, ids=ids.clone(), logits=logits.clone(), tau=2.0)
        got = [*c.fwd()]
        got += c.bwd(got[1])
        if want is None:
            want = got
            c.check()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), junk


def test_kept_entries_of_minus_infinity_and_the_lowest_value():
    x, w, dloss = head(5, 64, 300, 15)
    ids = torch.randint(0, 300, (5, 4), generator=gen(16)).to(I32)
    logits = torch.randn(5, 4, generator=gen(17))
    logits[0, 1] = -torch.inf
    logits[1] = -torch.inf                      # kept, but without a distribution
    logits[2, :3] = torch.finfo(torch.float32).min
    logits[3] = torch.finfo(torch.float32).min  # four equal entries
    c = Case(x, w, dloss, ids=ids, logits=logits)
    loss, _, dx, _ = c.check()
    assert loss[1] == 0 and not dx[1].any()


def test_a_broken_teacher_row_shows_and_stays_alone():
    x, w, dloss = head(4, 64, 300, 18)
    ids = torch.randint(0, 300, (4, 3), generator=gen(19)).to(I32)
    logits = torch.randn(4, 3, generator=gen(20))
    want, _ = Case(x, w, dloss, ids=ids, logits=logits).fwd()
    logits[2, 1] = float("nan")
    got, _ = Case(x, w, dloss, ids=ids, logits=logits).fwd()
    assert torch.isnan(got[2]) and torch.equal(got[[0, 1, 3]], want[[0, 1, 3]])


def test_large_logits_do_not_overflow():
    x, w, dloss = head(130, 64, 500, 21)
    t = torch.randint(0, 500, (130,), generator=gen(22)).to(I32)
    c = Case((x.float() * 100).to(BF16), w, dloss, targets=t)  # logits in the hundreds
    loss, lse, dx, dw = c.check()
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()


def test_either_gradient_alone():
    c = ce(150, 128, 700, seed=23)
    _, lse = c.fwd()
    dx, dw = c.bwd(lse)
    assert torch.equal(c.bwd(lse, dw=False)[0], dx)
    assert torch.equal(c.bwd(lse, dx=False)[1], dw)
    assert c.bwd(lse, dx=False, dw=False) == (None, None)


def test_no_rows():
    w = torch.ones(9, 64, dtype=BF16, device="cuda")
    x, t, s = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, dtype=I32, device="cuda"), torch.empty(
        0, device="cuda")
    ws = B.alloc_workspace(256)
    B.moe_lm_ce_fwd(x, w, t, s, s, ws)
    dw = torch.ones_like(w)
    B.moe_lm_ce_bwd(x, w, t, s, s, torch.empty_like(x), dw, ws)
    assert not dw.any()


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_several_pieces_of_the_vocabulary(kind):
    # 2 T V bytes pass the 512 MB of one piece, the last piece is shorter and ends inside a tile
    T, D, V = 16000, 64, 20001
    x, w, dloss = head(T, D, V, 24)
    dloss = dloss / T
    if kind == "ce":
        t = torch.randint(0, V, (T,), generator=gen(25)).to(I32)
        t[::7] = -100
        c = Case(x, w, dloss, targets=t)
    else:
        ids = torch.randint(0, V, (T, 6), generator=gen(25)).to(I32)
        ids[::9] = -1
        c = Case(x, w, dloss, ids=ids, logits=torch.randn(T, 6, generator=gen(26)), tau=2.0)
    loss, lse = c.fwd()
    dx, dw = c.bwd(lse)
    assert B.moe_get_status(c.ws) == 0
    d = c.dev
    sparse = c.sparse("cuda")
    wdw, bdw = torch.zeros(V, D, dtype=torch.double, device="cuda"), torch.zeros(V, D, dtype=torch.double, device="cuda")
    for a in range(0, T, 4000):  # rows at a time: the 64-bit logits of all would take 20 GB
        rows = slice(a, a + 4000)
        part = tuple(s[rows] for s in sparse)
        want = R.lm_fwd(d["x"][rows], d["w"], part, c.tau)
        R.check(loss[rows], want[0], want[2], "loss")
        R.check(lse[rows], want[1], want[3], "lse")
        rdx, rdw, bdx, b = R.lm_bwd(d["x"][rows], d["w"], part, lse[rows], d["dloss"][rows], c.tau)
        # this lse is the kernel's: its bound enters the exponent
        R.check(dx[rows], rdx, bdx, "dx")
        wdw += rdw
        bdw += b
    R.check(dw, wdw, bdw, "dw")


@pytest.mark.parametrize("T,D,V", [(520, 128, 5000), (513, 64, 129), (512, 1024, 4000), (8, 64, 9000), (120, 2048, 700)])
def test_gradients_in_one_grid_and_in_two(T, D, V):
    ce(T, D, V, seed=T + D + V).check()


def test_weights_past_32_bits():
    T, D, V = 3, 4096, 600_003  # over 2^31 elements of w and of dw
    w = torch.randn(V, D, device="cuda", dtype=BF16).mul_(2.0 / D ** 0.5)
    x = torch.randn(T, D, generator=gen(34)).to(BF16).cuda()
    dloss = torch.randn(T, generator=gen(35)).cuda()
    targets = torch.tensor([V - 1, 524_288, 7], dtype=I32, device="cuda")  # V - 1: its row is past 2^31
    ws = B.alloc_workspace(B.moe_lm_workspace_bytes(T, D, V))
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    B.moe_lm_ce_fwd(x, w, targets, loss, lse, ws)
    dx, dw = torch.empty_like(x), torch.full_like(w, 3.0)
    B.moe_lm_ce_bwd(x, w, targets, lse, dloss, dx, dw, ws)
    assert B.moe_get_status(ws) == 0
    z = torch.cat([x.double() @ w[a:a + 50_000].double().T for a in range(0, V, 50_000)], 1)
    # |x| |w| bounds the sum of a logit's absolute products; no row of w is longer than 3 (2 on average)
    dz = (D // 16 + 16) * R.ACC * x.double().norm(dim=1) * 3.0
    want = torch.logsumexp(z, 1)
    blse = dz + 8 * R.U32 * (z.abs().amax(1) + want.abs() + 2) + (300 + V // 4096) * R.U32
    R.check(lse, want, blse, "lse")
    zt = z.gather(1, targets.long()[:, None])[:, 0]
    R.check(loss, want - zt, 2 * blse + 8 * R.U32 * want.abs(), "loss")
    dl = dloss.double()[:, None] * torch.exp(z - lse.double()[:, None])
    dl[range(T), targets.long()] -= dloss.double()
    for rows in (slice(0, 300), slice(524_200, 524_400), slice(V - 300, V)):
        part = dl[:, rows]
        e = dz[:, None] + 8 * R.U32 * (z[:, rows].abs() + lse.double().abs()[:, None] + 2)
        bdl = (part.abs() + dloss.double().abs()[:, None] * 8 * R.U32) * e * 1.01 + R.round_bound(part, BF16)
        ref = part.T @ x.double()
        bound = (bdl.T @ x.double().abs()) * 1.01 + 80 * R.ACC * (part.abs().T @ x.double().abs()) + R.round_bound(ref, BF16)
        R.check(dw[rows], ref, bound, f"dw {rows}")
    assert torch.isfinite(dx.float()).all()


def test_repeats_and_another_stream_give_the_same_bits():
    c = distill(300, 256, 2000, 16, seed=27, tau=2.0)
    loss, lse = c.fwd()
    first = (loss, lse, *c.bwd(lse))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = (*c.fwd(stream=s), *c.bwd(lse, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_replay_with_new_inputs():
    a, b = ce(200, 128, 900, seed=28), ce(200, 128, 900, seed=40)
    want = []
    for c in (a, b):
        loss, lse = c.fwd()
        want.append((loss, lse, *c.bwd(lse)))
    d = {k: v.clone() for k, v in a.dev.items()}
    out = [torch.empty_like(t) for t in want[0]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_lm_ce_fwd(d["x"], d["w"], d["targets"], out[0], out[1], a.ws, stream=s)
        B.moe_lm_ce_bwd(d["x"], d["w"], d["targets"], out[1], d["dloss"], out[2], out[3], a.ws, stream=s)
    for c, ref in zip((a, b), want):
        for k in d:
            d[k].copy_(c.dev[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, ref))


def test_gradient_is_the_difference_of_the_forward():
    # W moves by whole bf16 steps along one direction, so that the moved weights are exact
    T, D, V = 64, 64, 300
    x, w, dloss = head(T, D, V, 30)
    t = torch.randint(0, V, (T,), generator=gen(31)).to(I32)
    dloss = dloss.abs() + 0.1
    w = (w.float() * 16).round().clamp(-8, 8).div(16).to(BF16)  # multiples of 1/16
    v = torch.randint(-1, 2, (V, D), generator=gen(32)).float()
    h = 1.0 / 64
    up, down = (Case(x, (w.float() + s * h * v).to(BF16), dloss, targets=t).fwd()[0].double() for s in (1, -1))
    diff = ((up - down) * dloss.cuda().double()).sum() / (2 * h)
    c = Case(x, w, dloss, targets=t)
    _, lse = c.fwd()
    _, dw = c.bwd(lse)
    got = (dw.double() * v.cuda().double()).sum()
    # the terms' bf16 roundings, and the third derivative of lse along v: |x.v|^3 of about D^1.5, over 6
    bound = float(dw.double().abs().sum()) * 2.0 ** -7 + T * D ** 1.5 * h * h + T * 2.0 ** -16 / h
    assert abs(float(diff - got)) < bound


def test_refusals():
    c = ce(8, 64, 30, seed=33)
    d, s = c.dev, torch.zeros(8, device="cuda")
    with pytest.raises(B.MoeError, match="WORKSPACE"):
        B.moe_lm_ce_fwd(d["x"], d["w"], d["targets"], s, s, c.ws[:256])
    with pytest.raises(ValueError, match="shape"):
        B.moe_lm_ce_fwd(d["x"], d["w"], d["targets"][:4], s, s, c.ws)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_lm_ce_fwd(d["x"], torch.zeros(30, 128, dtype=BF16, device="cuda")[:, :64], d["targets"], s, s, c.ws)
    with pytest.raises(TypeError):
        B.moe_lm_ce_bwd(d["x"], d["w"], d["targets"], s, s, d["x"].float(), None, c.ws)
