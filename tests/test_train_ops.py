"""The operators around the expert layer without a GPU: the 64-bit references against central
differences, refusals of the C entry points and of the binding, workspace sizes."""

import ctypes

import pytest
import torch

import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding, build

OK, INVALID, SHAPE, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
FAKE = 1 << 20  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def v(p):
    return ctypes.c_void_p(p)


# ------------------------------------------------------------- the references against differences

def differences(f, x, h=1e-6):
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + h
        up = f()
        flat[i] = keep - h
        down = f()
        flat[i] = keep
        out[i] = (up - down) / (2 * h)
    return g


def randn(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.double, generator=torch.Generator().manual_seed(seed))


def test_layernorm_gradients_are_the_differences():
    x, gamma, beta, dy = randn(3, 5, seed=1), 1 + 0.1 * randn(5, seed=2), randn(5, seed=3), randn(3, 5, seed=4)
    f = lambda: float((R.ln_fwd(x, gamma, beta, 1e-3)[0] * dy).sum())
    _, mean, rstd = R.ln_fwd(x, gamma, beta, 1e-3)
    dx, dgamma, dbeta = R.ln_bwd(dy, x, gamma, mean, rstd)
    for got, arg in ((dx, x), (dgamma, gamma), (dbeta, beta)):
        assert torch.allclose(got, differences(f, arg), atol=1e-7)


@pytest.mark.parametrize("normalize", [True, False])
def test_router_gradient_is_the_differences(normalize):
    z, ds = randn(4, 6, seed=5), randn(4, 3, seed=6)
    ids, _ = R.router_fwd(z, 3, normalize)
    f = lambda: float((R.router_fwd(z, 3, normalize)[1] * ds).sum())
    assert torch.allclose(R.router_bwd(z, ids, ds, normalize)[0], differences(f, z), atol=1e-8)


@pytest.mark.parametrize("kind", ["ce", "distill"])
def test_vocabulary_loss_gradients_are_the_differences(kind):
    T, D, V, tau = 4, 3, 7, 1.0 if kind == "ce" else 2.0
    x, w, dloss = randn(T, D, seed=7), randn(V, D, seed=8), randn(T, seed=9)
    if kind == "ce":
        target = R.sparse(targets=torch.tensor([0, 6, -100, 3]))
    else:
        ids = torch.tensor([[0, 1, 2], [6, 6, -1], [-1, -1, -1], [5, 4, 3]])
        target = R.sparse(teacher_ids=ids, teacher_logits=randn(T, 3, seed=10), tau=tau)
    f = lambda: float((R.lm_fwd(x, w, target, tau)[0] * dloss).sum())
    lse = torch.logsumexp(x @ w.T / tau, 1)
    dx, dw, _, _ = R.lm_bwd(x, w, target, lse, dloss, tau)
    assert torch.allclose(dx, differences(f, x), atol=1e-7)
    assert torch.allclose(dw, differences(f, w), atol=1e-7)


def test_cross_entropy_is_torchs():
    x, w = randn(6, 4, seed=11), randn(9, 4, seed=12)
    t = torch.tensor([0, 8, -100, 3, 3, -100])
    loss = R.lm_fwd(x, w, R.sparse(targets=t), 1.0)[0]
    assert torch.allclose(loss, torch.nn.functional.cross_entropy(x @ w.T, t, reduction="none"))


# ------------------------------------------------------------------------------------ C refusals

def test_layernorm_refusals(lib):
    fwd = lambda **k: lib.moe_layernorm_fwd(
        v(k.get("x", FAKE)), v(k.get("g", FAKE)), v(FAKE), k.get("dt", 1), k.get("pt", 0), v(k.get("y", FAKE)),
        v(k.get("mean", FAKE)), v(FAKE), k.get("T", 4), k.get("D", 8), ctypes.c_float(k.get("eps", 1e-5)), None)
    assert fwd(T=0) == OK
    assert fwd(T=0, x=0, y=0) == OK
    assert fwd(T=-1) == INVALID
    assert fwd(D=0) == INVALID
    assert fwd(dt=3) == INVALID
    assert fwd(pt=-1) == INVALID
    assert fwd(eps=-1.0) == INVALID
    assert fwd(eps=float("nan")) == INVALID
    assert fwd(x=0) == INVALID
    assert fwd(mean=0) == INVALID
    assert fwd(T=1 << 31) == SHAPE
    assert fwd(D=(1 << 24) + 1) == SHAPE
    assert fwd(x=FAKE + 1) == MISALIGNED
    assert fwd(dt=0, y=FAKE + 2) == MISALIGNED
    assert fwd(g=FAKE + 2) == MISALIGNED  # 32-bit parameters
    need = binding.moe_layernorm_bwd_workspace_bytes(4, 8)
    bwd = lambda **k: lib.moe_layernorm_bwd(
        v(k.get("dy", FAKE)), v(FAKE), v(0), v(FAKE), v(k.get("rstd", FAKE)), k.get("dt", 2), k.get("pt", 2),
        v(k.get("dx", FAKE)), v(k.get("dg", FAKE)), v(FAKE), k.get("T", 4), k.get("D", 8), v(k.get("ws", FAKE)),
        k.get("wsb", need), None)
    assert bwd(T=-1) == INVALID
    assert bwd(dy=0) == INVALID
    assert bwd(rstd=0) == INVALID
    assert bwd(dx=0) == INVALID
    assert bwd(ws=0) == INVALID
    assert bwd(dt=9) == INVALID
    assert bwd(dx=FAKE + 1) == MISALIGNED
    assert bwd(dg=FAKE + 1) == MISALIGNED
    assert bwd(ws=FAKE + 16) == MISALIGNED
    assert bwd(wsb=need - 1) == WS_SMALL
    assert binding.moe_layernorm_bwd_workspace_bytes(0, 8) == 0
    assert binding.moe_layernorm_bwd_workspace_bytes(4, 0) == 0


def test_router_refusals(lib):
    fwd = lambda **k: lib.moe_router_topk_fwd(
        v(k.get("z", FAKE)), k.get("dt", 0), v(k.get("ids", FAKE)), v(FAKE), k.get("T", 4), k.get("E", 8),
        k.get("K", 2), 1, None)
    bwd = lambda **k: lib.moe_router_topk_bwd(
        v(k.get("z", FAKE)), k.get("dt", 0), v(k.get("ids", FAKE)), v(k.get("ds", FAKE)), v(k.get("dz", FAKE)),
        k.get("T", 4), k.get("E", 8), k.get("K", 2), 0, None)
    for call in (fwd, bwd):
        assert call(T=0) == OK
        assert call(T=-1) == INVALID
        assert call(E=0) == INVALID
        assert call(K=0) == INVALID
        assert call(K=9) == INVALID
        assert call(dt=2) == INVALID
        assert call(z=0) == INVALID
        assert call(ids=0) == INVALID
        assert call(E=4097) == SHAPE
        assert call(z=FAKE + 2) == MISALIGNED
        assert call(ids=FAKE + 2) == MISALIGNED
    assert bwd(ds=0) == INVALID
    assert bwd(dz=0) == INVALID
    assert bwd(dz=FAKE + 2) == MISALIGNED


def test_vocabulary_loss_refusals(lib):
    f = ctypes.c_float
    need = binding.moe_lm_workspace_bytes(4, 64, 10, 3)
    d = dict(x=FAKE, w=FAKE, t=FAKE, tl=FAKE, tau=1.0, a=FAKE, b=FAKE, dx=FAKE, dw=FAKE, T=4, D=64, V=10, K=3, ws=FAKE,
             wsb=need)
    calls = {
        "ce_fwd": lambda a: lib.moe_lm_ce_fwd(v(a["x"]), v(a["w"]), v(a["t"]), -100, v(a["a"]), v(a["b"]), a["T"],
                                              a["D"], a["V"], v(a["ws"]), a["wsb"], None),
        "ce_bwd": lambda a: lib.moe_lm_ce_bwd(v(a["x"]), v(a["w"]), v(a["t"]), -100, v(a["a"]), v(a["b"]), v(a["dx"]),
                                              v(a["dw"]), a["T"], a["D"], a["V"], v(a["ws"]), a["wsb"], None),
        "distill_fwd": lambda a: lib.moe_lm_distill_fwd(
            v(a["x"]), v(a["w"]), v(a["t"]), v(a["tl"]), f(a["tau"]), v(a["a"]), v(a["b"]), a["T"], a["D"], a["V"],
            a["K"], v(a["ws"]), a["wsb"], None),
        "distill_bwd": lambda a: lib.moe_lm_distill_bwd(
            v(a["x"]), v(a["w"]), v(a["t"]), v(a["tl"]), f(a["tau"]), v(a["a"]), v(a["b"]), v(a["dx"]), v(a["dw"]),
            a["T"], a["D"], a["V"], a["K"], v(a["ws"]), a["wsb"], None),
    }
    for name, fn in calls.items():
        call = lambda **k: fn({**d, **k})
        assert call(T=-1) == INVALID, name
        assert call(D=0) == INVALID
        assert call(V=0) == INVALID
        assert call(x=0) == INVALID
        assert call(w=0) == INVALID
        assert call(t=0) == INVALID
        assert call(a=0) == INVALID
        assert call(b=0) == INVALID
        assert call(ws=0) == INVALID
        assert call(D=72) == SHAPE
        assert call(V=(1 << 30) + 1) == SHAPE
        assert call(T=1 << 31) == SHAPE
        assert call(x=FAKE + 8) == MISALIGNED
        assert call(w=FAKE + 2) == MISALIGNED
        assert call(t=FAKE + 2) == MISALIGNED
        assert call(a=FAKE + 1) == MISALIGNED
        assert call(ws=FAKE + 128) == MISALIGNED
        assert call(wsb=1) == WS_SMALL
        if name.startswith("distill"):
            assert call(K=0) == INVALID
            assert call(K=257) == SHAPE
            assert call(tl=0) == INVALID
            assert call(wsb=need - 1) == WS_SMALL
            for tau in (0.0, -1.0, float("inf"), float("nan")):
                assert call(tau=tau) == INVALID
        if name.endswith("bwd"):
            assert call(dx=FAKE + 8) == MISALIGNED
            assert call(dw=FAKE + 8) == MISALIGNED
            assert call(dx=0, dw=0) == OK  # nothing asked for
        else:
            assert call(T=0) == OK


def test_vocabulary_workspace_does_not_grow_with_the_logits(lib):
    size = binding.moe_lm_workspace_bytes
    assert size(0, 64, 10) == 0 and size(4, 65, 10) == 0 and size(4, 64, 0) == 0 and size(4, 64, 10, 257) == 0
    assert size(1, 64, 1) > 0
    assert size(1 << 25, 64, 1 << 18) == 0  # 2^28 tiles of logits
    T, D, V = 32768, 4096, 131072
    logits = 2 * T * V
    assert size(T, D, V) < logits // 4
    assert size(T, D, 2 * V) - size(T, D, V) < logits // 100
    assert size(T, D, V, 64) - size(T, D, V, 1) <= 12 * 64 * T


# ------------------------------------------------------------------------------ binding refusals

def test_binding_refuses_what_the_kernels_do_not_take():
    bf, i32 = torch.bfloat16, torch.int32
    x, y, s = torch.zeros(4, 8, dtype=bf), torch.zeros(4, 8, dtype=bf), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_layernorm_fwd(x, None, None, y, s, s)
    with pytest.raises(TypeError):
        binding.moe_layernorm_fwd(x.int(), None, None, y, s, s)
    with pytest.raises(ValueError, match="dims"):
        binding.moe_layernorm_fwd(x[0], None, None, y, s, s)
    with pytest.raises(TypeError):
        binding.moe_router_topk_fwd(torch.zeros(4, 8, dtype=torch.float16), torch.zeros(4, 2, dtype=i32), s)
    with pytest.raises(TypeError):
        binding.moe_lm_ce_fwd(x.float(), y, torch.zeros(4, dtype=i32), s, s, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_lm_distill_fwd(x, y, torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2), s, s,
                                   torch.zeros(8, dtype=torch.uint8))
