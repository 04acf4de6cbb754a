"""Layer norm on the GPU against its 64-bit values, within the rounding each type allows: lengths on both
sides of every kernel's range, rows that do not start on 16-byte boundaries, all types, absent parameters."""

import pytest
import torch

import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def rand(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype)


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def fwd(x, gamma, beta, eps=1e-5, y=None, stream=None):
    T, D = x.shape
    y = torch.empty_like(x) if y is None else y
    mean, rstd = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    B.moe_layernorm_fwd(x, gamma, beta, y, mean, rstd, eps, stream=stream)
    return y, mean, rstd


def bwd(dy, x, gamma, mean, rstd, param_dtype, stream=None):
    T, D = x.shape
    ws = B.alloc_workspace(B.moe_layernorm_bwd_workspace_bytes(T, D))
    dx = torch.full_like(x, 3.0)
    dgamma, dbeta = (torch.full((D,), 3.0, dtype=param_dtype, device="cuda") for _ in range(2))
    B.moe_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, stream=stream)
    return dx, dgamma, dbeta


def compare_fwd(x, gamma, beta, eps=1e-5):
    got = fwd(*cuda(x, gamma, beta), eps)
    for name, a, b, c in zip(("y", "mean", "rstd"), got, R.ln_fwd(x, gamma, beta, eps),
                             R.ln_fwd_bounds(x, gamma, beta, eps, x.dtype)):
        R.check(a, b, c, name)


def compare_bwd(dy, x, gamma, param_dtype, eps=1e-5):
    _, mean, rstd = (t.float() for t in R.ln_fwd(x, gamma, None, eps))
    got = bwd(*cuda(dy, x, gamma, mean, rstd), param_dtype)
    for name, a, b, c in zip(("dx", "dgamma", "dbeta"), got, R.ln_bwd(dy, x, gamma, mean, rstd),
                             R.ln_bwd_bounds(dy, x, gamma, mean, rstd, x.dtype, param_dtype)):
        R.check(a, b, c, name)


LENGTHS = [(1, 1), (1, 8), (3, 7), (5, 256), (6, 257), (130, 264), (9, 512), (7, 520), (3, 1001), (4, 1024), (5, 1032),
           (2, 2048), (3, 2056), (3, 4096), (2, 4104), (2, 7168), (3, 8191), (2, 8192), (3, 8200), (2, 20001)]


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,D", LENGTHS)
def test_forward(T, D, dtype):
    seed = T * 10007 + D
    x = rand(T, D, seed=seed, dtype=dtype, shift=0.5)
    compare_fwd(x, rand(D, seed=seed + 1, dtype=dtype, shift=1.0), rand(D, seed=seed + 2, dtype=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,D", LENGTHS + [(700, 64), (1300, 513), (700, 2048), (400, 8200)])
def test_backward(T, D, dtype):
    seed = T * 10007 + D
    compare_bwd(rand(T, D, seed=seed, dtype=dtype), rand(T, D, seed=seed + 1, dtype=dtype, shift=0.5),
                rand(D, seed=seed + 2, dtype=dtype, shift=1.0), dtype)


@pytest.mark.parametrize("dtype,param", [(BF16, F32), (F16, F32), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("D", [72, 1001, 2048, 9000])
def test_parameters_of_another_type(D, dtype, param):
    x, gamma, beta = rand(5, D, seed=D, dtype=dtype), rand(D, seed=D + 1, dtype=param), rand(D, seed=D + 2, dtype=param)
    compare_fwd(x, gamma, beta)
    compare_bwd(rand(5, D, seed=D + 3, dtype=dtype), x, gamma, param)


def test_without_parameters():
    x = rand(9, 200, seed=1, dtype=BF16)
    compare_fwd(x, None, None)
    compare_fwd(x, rand(200, seed=2), None)
    compare_fwd(x, None, rand(200, seed=2))
    compare_bwd(rand(9, 200, seed=3, dtype=BF16), x, None, F32)


def test_each_parameter_gradient_alone_and_none():
    dy, x = rand(40, 96, seed=1), rand(40, 96, seed=2)
    _, mean, rstd = (t.float() for t in R.ln_fwd(x, None, None, 1e-5))
    dy, x, mean, rstd = cuda(dy, x, mean, rstd)
    dx0, dg0, db0 = bwd(dy, x, None, mean, rstd, F32)
    ws = B.alloc_workspace(B.moe_layernorm_bwd_workspace_bytes(40, 96))
    dx, dg, db = torch.empty_like(x), torch.empty(96, device="cuda"), torch.empty(96, device="cuda")
    B.moe_layernorm_bwd(dy, x, None, mean, rstd, dx, dg, None, ws)
    assert torch.equal(dx, dx0) and torch.equal(dg, dg0)
    B.moe_layernorm_bwd(dy, x, None, mean, rstd, dx, None, db, ws)
    assert torch.equal(db, db0)
    dx.zero_()
    B.moe_layernorm_bwd(dy, x, None, mean, rstd, dx, None, None, None)
    assert torch.equal(dx, dx0)


def test_a_large_mean_does_not_cancel_the_variance():
    x = rand(4, 1000, seed=5, shift=1000.0)
    compare_fwd(x, None, None)


def test_constant_rows():
    x = torch.full((3, 640), 2.5)
    y, mean, rstd = fwd(x.cuda(), None, None, 1e-5)
    assert torch.equal(y.cpu(), torch.zeros(3, 640)) and torch.equal(mean.cpu(), x[:, 0])
    assert torch.allclose(rstd.cpu(), torch.full((3,), 1e-5 ** -0.5))


def test_one_bad_row_stays_alone():
    x = rand(6, 512, seed=6)
    x[2, 5] = float("nan")
    x[4, 0] = float("inf")
    y, _, _ = fwd(x.cuda(), None, None)
    clean, _, _ = fwd(x[[0, 1, 3, 5]].cuda(), None, None)
    assert torch.equal(y[[0, 1, 3, 5]], clean)
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()


@pytest.mark.parametrize("D", [96, 1001, 4096, 8200])
def test_in_place(D):
    x, dy = rand(33, D, seed=7, dtype=BF16).cuda(), rand(33, D, seed=8, dtype=BF16).cuda()
    y, mean, rstd = fwd(x, None, None)
    z = x.clone()
    fwd(z, None, None, y=z)
    assert torch.equal(z, y)
    dx, dg, db = bwd(dy, x, None, mean, rstd, F32)
    ws = B.alloc_workspace(B.moe_layernorm_bwd_workspace_bytes(33, D))
    dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
    for out in (dy.clone(), x.clone()):
        first = out.data_ptr()
        a, b = (out, x) if torch.equal(out, dy) else (dy, out)
        B.moe_layernorm_bwd(a, b, None, mean, rstd, out, dg2, db2, ws)
        assert out.data_ptr() == first and torch.equal(out, dx) and torch.equal(dg2, dg) and torch.equal(db2, db)


def test_a_view_that_starts_off_the_boundary():
    base = rand(5 * 640 + 3, seed=9, dtype=BF16).cuda()
    x = base[3:].view(5, 640)
    y, _, _ = fwd(x, None, None)
    want, _, _ = fwd(x.clone(), None, None)
    assert torch.allclose(y.float(), want.float(), atol=0.02)
    R.check(y, R.ln_fwd(x.cpu(), None, None, 1e-5)[0], R.ln_fwd_bounds(x.cpu(), None, None, 1e-5, BF16)[0])


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = fwd(x, None, None)
    dx, dgamma, dbeta = bwd(x, x, None, mean, rstd, F32)
    assert not dgamma.any() and not dbeta.any()


def test_refuses_strided_rows():
    x = torch.zeros(8, 64, device="cuda")[:, :32]
    with pytest.raises(ValueError, match="contiguous"):
        fwd(x, None, None)


def test_repeats_and_another_stream_give_the_same_bits():
    dy, x = rand(3000, 640, seed=11, dtype=BF16).cuda(), rand(3000, 640, seed=12, dtype=BF16).cuda()
    _, mean, rstd = fwd(x, None, None)
    first = bwd(dy, x, None, mean, rstd, F32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = bwd(dy, x, None, mean, rstd, F32, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradient_is_the_difference_of_the_forward():
    T, D, h = 4, 96, 1e-2
    x, v, dy = (rand(T, D, seed=s) for s in (13, 14, 15))
    x, v, dy = cuda(x, v, dy)
    up, down = (fwd(x + s * h * v, None, None)[0].double() for s in (1, -1))
    _, mean, rstd = fwd(x, None, None)
    dx, _, _ = bwd(dy, x, None, mean, rstd, F32)
    diff = ((up - down) * dy.double()).sum() / (2 * h)
    # the difference's own error: h^2 third derivatives of O(1) per element, and fp32 values over 2 h
    assert abs(float(diff - (dx.double() * v.double()).sum())) < T * D * (h * h + 2.0 ** -22 / h)


def test_offsets_past_32_bits():
    T, D = 300_001, 7168  # over 2^31 elements
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    rows = [0, 149_797, 299_593, T - 1]  # both sides of 2^30 and of 2^31 elements
    x[rows] = rand(len(rows), D, seed=18, dtype=BF16).cuda()
    y, mean, rstd = fwd(x, None, None)
    want, wmean, wrstd = fwd(x[rows].contiguous(), None, None)
    assert torch.equal(y[rows], want) and torch.equal(mean[rows], wmean) and torch.equal(rstd[rows], wrstd)
    assert not y[rows[1] + 1].any()
    del y
    dx, dg, db = bwd(x, x, None, mean, rstd, F32)
    wdx, wdg, wdb = bwd(x[rows].contiguous(), x[rows].contiguous(), None, wmean, wrstd, F32)
    assert torch.equal(dx[rows], wdx)
    # the other rows add nothing: the same terms, added in another order
    terms = (x[rows].double().abs() * ((x[rows].double() - wmean[:, None]) * wrstd[:, None]).abs()).sum(0)
    assert ((dg - wdg).abs() <= 16 * R.U32 * terms).all()
    assert ((db - wdb).abs() <= 16 * R.U32 * x[rows].double().abs().sum(0)).all()


def test_graph_replay():
    dy, x = rand(50, 640, seed=16, dtype=BF16).cuda(), rand(50, 640, seed=17, dtype=BF16).cuda()
    y, mean, rstd = fwd(x, None, None)
    dx, dg, db = bwd(dy, x, None, mean, rstd, F32)
    ws = B.alloc_workspace(B.moe_layernorm_bwd_workspace_bytes(50, 640))
    out = [torch.empty_like(t) for t in (y, mean, rstd, dx, dg, db)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_layernorm_fwd(x, None, None, *out[:3], stream=s)
        B.moe_layernorm_bwd(dy, x, None, out[1], out[2], *out[3:], ws, stream=s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (y, mean, rstd, dx, dg, db)))
