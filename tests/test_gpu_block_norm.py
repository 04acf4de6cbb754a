"""The norms around a block on the GPU against their 64-bit values, within the rounding each type allows: lengths on
both sides of every kernel's range, rows that do not start on 16-byte boundaries, all types, every combination of
norm, gate and parameters."""

import itertools

import pytest
import torch

import block_norm_ref as N
import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-6


def rand(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def make(T, D, dtype, param, post=True, gate="channel", gammas=True, seed=0):
    seed = 100 * seed + 7 * T + D
    c = dict(block=rand(T, D, seed=seed, dtype=dtype), residual=rand(T, D, seed=seed + 1, dtype=dtype, scale=2.0),
             post_gamma=rand(D, seed=seed + 2, dtype=param, scale=0.3, shift=1.0) if post and gammas else None,
             pre_gamma=rand(D, seed=seed + 3, dtype=param, scale=0.3, shift=1.0) if gammas else None, gate=None)
    if gate == "channel":
        c["gate"] = rand(D, seed=seed + 4, dtype=param, shift=0.5)
    elif gate == "token":
        c["gate"] = rand(T, D, seed=seed + 4, dtype=dtype, shift=0.5)
    return c


def fwd(c, post, scale, stream_out=None, normed=None, stream=None):
    block, residual, post_gamma, gate, pre_gamma = cuda(*(c[k] for k in ("block", "residual", "post_gamma", "gate",
                                                                       "pre_gamma")))
    T = block.shape[0]
    stream_out = torch.full_like(block, 7.0) if stream_out is None else stream_out
    normed = torch.full_like(block, 7.0) if normed is None else normed
    post_rstd = torch.full((T,), 7.0, device="cuda") if post else None
    pre_rstd = torch.full((T,), 7.0, device="cuda")
    B.moe_block_norm_fwd(block, residual, post_gamma, gate, pre_gamma, stream_out, normed, post_rstd, pre_rstd,
                         residual_scale=scale, eps=EPS, stream=stream)
    return stream_out, normed, post_rstd, pre_rstd


def compare_fwd(c, post, scale=0.7):
    got = fwd(c, post, scale)
    want = N.fwd(*(c[k] for k in ("block", "residual", "post_gamma", "gate", "pre_gamma")), scale, EPS, post)
    bounds = N.fwd_bounds(*(c[k] for k in ("block", "residual", "post_gamma", "gate", "pre_gamma")), scale, EPS, post,
                          c["block"].dtype)
    for name, g, w, b in zip(("stream", "normed", "post_rstd", "pre_rstd"), got, want, bounds):
        assert (g is None) == (w is None)
        if g is not None:
            R.check(g, w, b, name)


NAMES = ("dblock", "dresidual", "dpost_gamma", "dgate", "dpre_gamma")


def back(c, param, post, scale, dstream=True, want=NAMES, seed=50, out=None, stream=None):
    """The inputs on the host, and the gradients that the kernels make."""
    T, D = c["block"].shape
    dtype = c["block"].dtype
    s, _, post_rstd, pre_rstd, _ = N.fwd(c["block"], c["residual"], c["post_gamma"], c["gate"], c["pre_gamma"], scale,
                                         EPS, post)
    a = dict(dstream=rand(T, D, seed=seed, dtype=dtype) if dstream else None, dnormed=rand(T, D, seed=seed + 1, dtype=dtype),
             block=c["block"] if post or c["gate"] is not None else None, stream=s.to(dtype),
             post_gamma=c["post_gamma"], gate=c["gate"], pre_gamma=c["pre_gamma"],
             post_rstd=None if post_rstd is None else post_rstd.float(), pre_rstd=pre_rstd.float())
    dev = cuda(*a.values())
    blank = lambda shape, dt: torch.full(shape, 3.0, dtype=dt, device="cuda")
    g = {"dblock": blank((T, D), dtype), "dresidual": blank((T, D), dtype), "dpost_gamma": None, "dgate": None,
         "dpre_gamma": None}
    if post and "dpost_gamma" in want:
        g["dpost_gamma"] = blank((D,), param)
    if c["gate"] is not None and "dgate" in want:
        g["dgate"] = blank(c["gate"].shape, c["gate"].dtype)
    if "dpre_gamma" in want:
        g["dpre_gamma"] = blank((D,), param)
    if out:
        g.update({k: dev[list(a).index(v)] for k, v in out.items()})
    sums = any(g[k] is not None and g[k].dim() == 1 for k in NAMES[2:])
    ws = B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(T, D)) if sums else None
    if ws is not None:
        ws.fill_(0xFF)  # not a number, whatever it is read as
    B.moe_block_norm_bwd(*dev, *(g[k] for k in NAMES), ws, residual_scale=scale, stream=stream)
    return a, g


def compare_bwd(c, param, post, scale=0.7, dstream=True):
    a, got = back(c, param, post, scale, dstream)
    want, bounds = N.bwd(*a.values(), scale)
    for name, w, e in zip(NAMES, want, bounds):
        g = got[name]
        assert (g is None) == (w is None), name
        if g is not None:
            R.check(g, w, e + R.round_bound(w, g.dtype), name)


LENGTHS = [(1, 1), (1, 8), (3, 7), (5, 256), (6, 257), (130, 264), (9, 512), (7, 520), (3, 1001), (4, 1024), (5, 1032),
           (2, 2048), (3, 2056), (3, 4096), (2, 4104), (2, 7168), (3, 8191), (2, 8192), (3, 8200), (2, 20001)]
TYPES = pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])


@TYPES
@pytest.mark.parametrize("T,D", LENGTHS + [(700, 96), (333, 4096)])
def test_forward(T, D, dtype):
    compare_fwd(make(T, D, dtype, dtype), True)
    compare_fwd(make(T, D, dtype, dtype, gate="token"), True)


@TYPES
@pytest.mark.parametrize("T,D", LENGTHS + [(700, 64), (1300, 513), (700, 2048), (400, 8200), (320, 13000)])
def test_backward(T, D, dtype):
    compare_bwd(make(T, D, dtype, dtype), dtype, True)
    compare_bwd(make(T, D, dtype, dtype, gate="token"), dtype, True)


COMBINATIONS = list(itertools.product([True, False], ["none", "channel", "token"], [True, False], [True, False]))


@pytest.mark.parametrize("D", [72, 1001, 9000])
@pytest.mark.parametrize("post,gate,gammas,dstream", COMBINATIONS)
def test_every_combination(D, post, gate, gammas, dstream):
    c = make(6, D, BF16, F32, post, gate, gammas)
    compare_fwd(c, post)
    compare_bwd(c, F32, post, dstream=dstream)


@pytest.mark.parametrize("dtype,param", [(BF16, F32), (F16, F32), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("D", [72, 1001, 2048, 9000])
def test_parameters_of_another_type(D, dtype, param):
    c = make(5, D, dtype, param)
    compare_fwd(c, True)
    compare_bwd(c, param, True)


@pytest.mark.parametrize("scale", [0.0, -1.5, 1.0])
def test_residual_scales(scale):
    c = make(40, 640, BF16, F32, gate="token")
    compare_fwd(c, True, scale)
    compare_bwd(c, F32, True, scale)


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_each_gradient_alone_and_none(gate):
    c = make(40, 96, F32, F32, gate=gate)
    _, full = back(c, F32, True, 1.0)
    for want in ((), ("dpost_gamma",), ("dgate",), ("dpre_gamma",)):
        _, some = back(c, F32, True, 1.0, want=want)
        for name in NAMES:
            if some[name] is not None:
                assert torch.equal(some[name], full[name]), (want, name)


def test_against_two_layer_steps():
    """The same as the pieces that a program without it would run, in torch's own rms_norm."""
    c = make(9, 320, F32, F32)
    b, r, pg, g, qg = cuda(c["block"], c["residual"], c["post_gamma"], c["gate"], c["pre_gamma"])
    stream, normed, _, _ = fwd(c, True, 0.7)
    want = 0.7 * r + g * torch.nn.functional.rms_norm(b, (320,), pg, EPS)
    assert torch.allclose(stream, want, rtol=1e-5, atol=1e-6)
    assert torch.allclose(normed, torch.nn.functional.rms_norm(want, (320,), qg, EPS), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("dtype,D", [(BF16, 96), (BF16, 1001), (BF16, 4096), (F32, 8200)])
def test_in_place(dtype, D):
    c = make(33, D, dtype, dtype)
    want = fwd(c, True, 0.7)
    for stream_is, normed_is in (("residual", "block"), ("block", "residual"), ("residual", None), (None, "block")):
        d = dict(c, block=c["block"].cuda(), residual=c["residual"].cuda())
        got = fwd(d, True, 0.7, stream_out=d.get(stream_is), normed=d.get(normed_is))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (stream_is, normed_is)
    _, want = back(c, dtype, True, 0.7)
    for dblock, dresidual in (("dnormed", "dstream"), ("block", "stream"), ("stream", "dnormed")):
        _, got = back(c, dtype, True, 0.7, out={"dblock": dblock, "dresidual": dresidual})
        assert all(torch.equal(got[k], want[k]) for k in NAMES), (dblock, dresidual)


def test_views_that_start_off_the_boundary():
    c = make(5, 640, BF16, BF16)
    want = fwd(c, True, 1.0)
    for name in ("block", "residual"):
        base = torch.empty(5 * 640 + 3, dtype=BF16, device="cuda")
        base[3:] = c[name].cuda().view(-1)
        got = fwd(dict(c, **{name: base[3:].view(5, 640)}), True, 1.0)
        for a, b in zip(got[:2], N.fwd(*(c[k] for k in ("block", "residual", "post_gamma", "gate", "pre_gamma")), 1.0, EPS,
                                       True)):
            assert float((a.cpu().double() - b).abs().max()) <= 2.0 ** -8 * float(b.abs().max())
        assert torch.allclose(got[3], want[3], rtol=1e-6)


def test_zero_and_huge_rows():
    c = make(4, 512, F32, F32)
    c["block"][1], c["residual"][1] = 0.0, 0.0
    c["block"][2] *= 1e15
    compare_fwd(c, True)
    compare_bwd(c, F32, True)


def test_one_bad_row_stays_alone():
    c = make(6, 512, F32, F32)
    c["block"][2, 5], c["residual"][4, 0] = float("nan"), float("inf")
    got = fwd(c, True, 1.0)
    keep = [0, 1, 3, 5]
    clean = fwd(dict(c, block=c["block"][keep], residual=c["residual"][keep]), True, 1.0)
    assert all(torch.equal(a[keep], b) for a, b in zip(got, clean))
    assert torch.isnan(got[1][2]).all() and torch.isnan(got[1][4, 0])


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    e = torch.empty(0, device="cuda")
    B.moe_block_norm_fwd(x, x, None, None, None, x, x, e, e)
    grads = [torch.full((64,), 3.0, device="cuda") for _ in range(3)]
    B.moe_block_norm_bwd(x, x, x, x, None, grads[0], None, e, e, x, x, *grads, None)
    assert not any(g.any() for g in grads)


def test_refuses_strided_rows():
    x = torch.zeros(8, 64, device="cuda")[:, :32]
    e = torch.empty(8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_block_norm_fwd(x, x, None, None, None, x, x, e, e)
    y = torch.zeros(8, 32, device="cuda")
    with pytest.raises(ValueError, match="gate"):
        B.moe_block_norm_fwd(y, y, None, x, None, y, y.clone(), e, e)


def test_repeats_and_another_stream_give_the_same_bits():
    c = make(3000, 640, BF16, F32)
    first = fwd(c, True, 1.0), back(c, F32, True, 1.0)[1]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = fwd(c, True, 1.0, stream=s), back(c, F32, True, 1.0, stream=s)[1]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first[0], again[0]))
    assert all(torch.equal(first[1][k], again[1][k]) for k in NAMES)


def test_gradient_is_the_difference_of_the_forward():
    T, D, h = 4, 96, 1e-2
    c = make(T, D, F32, F32)
    vb, vr = rand(T, D, seed=61), rand(T, D, seed=62)
    a, g = back(c, F32, True, 0.7)
    ends = []
    for sign in (1, -1):
        s, n, _, _ = fwd(dict(c, block=c["block"] + sign * h * vb, residual=c["residual"] + sign * h * vr), True, 0.7)
        ends.append((s.double().cpu() * a["dstream"].double()).sum() + (n.double().cpu() * a["dnormed"].double()).sum())
    diff = (ends[0] - ends[1]) / (2 * h)
    dot = (g["dblock"].cpu().double() * vb.double()).sum() + (g["dresidual"].cpu().double() * vr.double()).sum()
    # the difference's own error: h^2 third derivatives of O(1) per element, and fp32 values over 2 h
    assert abs(float(diff - dot)) < 4 * T * D * (h * h + 2.0 ** -22 / h)


def test_offsets_past_32_bits():
    T, D = 300_001, 7168  # over 2^31 elements
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    rows = [0, 149_797, 299_593, T - 1]
    x[rows] = rand(len(rows), D, seed=18, dtype=BF16).cuda()
    f = lambda n: torch.empty(n, device="cuda")
    stream, post, pre = torch.empty_like(x), f(T), f(T)
    B.moe_block_norm_fwd(x, x, None, None, None, stream, x, post, pre)  # normed over the inputs
    small = rand(len(rows), D, seed=18, dtype=BF16).cuda()
    ws, wn, wpost, wpre = torch.empty_like(small), torch.empty_like(small), f(4), f(4)
    B.moe_block_norm_fwd(small, small, None, None, None, ws, wn, wpost, wpre)
    assert torch.equal(stream[rows], ws) and torch.equal(x[rows], wn) and torch.equal(pre[rows], wpre)
    assert not x[rows[1] + 1].any()
    dpre, wdpre = f(D), f(D)
    space = B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(T, D))
    wdb, wdr = torch.empty_like(small), torch.empty_like(small)
    B.moe_block_norm_bwd(None, wn, wn, ws, None, None, None, wpost, wpre, wdb, wdr, None, None, wdpre, space)
    B.moe_block_norm_bwd(None, x, x, stream, None, None, None, post, pre, stream, x, None, None, dpre, space)
    assert torch.equal(stream[rows], wdb) and torch.equal(x[rows], wdr)
    # the other rows add nothing: the same terms, added in another order
    terms = (wn.double().abs() * ws.double().abs() * wpre.double()[:, None]).sum(0)
    assert ((dpre - wdpre).abs() <= 16 * R.U32 * terms).all()


def test_graph_replay():
    c = make(50, 640, BF16, F32)
    d = {k: v.cuda() for k, v in c.items()}
    args = (d["post_gamma"], d["gate"], d["pre_gamma"])
    want = fwd(c, True, 1.0)
    st, no, post, pre = (torch.empty_like(t) for t in want)
    ws = B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(50, 640))
    grads = [torch.empty_like(st), torch.empty_like(st)] + [torch.empty(640, device="cuda") for _ in range(3)]
    run_bwd = lambda g, s=None: B.moe_block_norm_bwd(d["residual"], d["block"], d["block"], st, *args, post, pre, *g, ws,
                                                     stream=s)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_block_norm_fwd(d["block"], d["residual"], *args, st, no, post, pre, stream=s)
        run_bwd(grads, s)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    eager = [torch.empty_like(t) for t in grads]
    run_bwd(eager)
    assert all(torch.equal(a, b) for a, b in zip((st, no, post, pre), want))
    assert all(torch.equal(a, b) for a, b in zip(grads, eager))
