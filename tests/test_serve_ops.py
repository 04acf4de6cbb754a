"""The norms around a block and the operators of a decoding step without a GPU: the 64-bit references against central
differences, refusals of the C entry points and of the binding, workspace sizes."""

import ctypes

import pytest
import torch

import block_norm_ref as N
from mixture_experts_routed_topk_gb300 import binding, build
from test_train_ops import differences, randn
from test_train_ops_calls import FAKE, Library, Stream, WRAP, tensor

OK, INVALID, SHAPE, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def v(p):
    return ctypes.c_void_p(p)


def f(x):
    return ctypes.c_float(x)


# ------------------------------------------------------------------------------ norms around a block

@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradients_are_the_differences(gate, post):
    T, D, scale, eps = 3, 5, 0.6, 1e-3
    c = dict(block=randn(T, D, seed=1), residual=randn(T, D, seed=2), post_gamma=1 + 0.1 * randn(D, seed=3) if post else None,
             gate={"none": None, "channel": randn(D, seed=4), "token": randn(T, D, seed=4)}[gate],
             pre_gamma=1 + 0.1 * randn(D, seed=5))
    ds, dn = randn(T, D, seed=6), randn(T, D, seed=7)

    def loss():
        s, n, _, _, _ = N.fwd(*c.values(), scale, eps, post)
        return float((s * ds).sum() + (n * dn).sum())

    s, _, post_rstd, pre_rstd, _ = N.fwd(*c.values(), scale, eps, post)
    got, _ = N.bwd(ds, dn, c["block"], s, c["post_gamma"], c["gate"], c["pre_gamma"], post_rstd, pre_rstd, scale)
    for grad, name in zip(got, ("block", "residual", "post_gamma", "gate", "pre_gamma")):
        assert (grad is None) == (c[name] is None)
        if grad is not None:
            assert torch.allclose(grad, differences(loss, c[name]), atol=1e-7), name


def test_block_norm_refusals(lib):
    fwd = lambda **k: lib.moe_block_norm_fwd(
        v(k.get("b", FAKE)), v(k.get("r", FAKE)), v(k.get("pg", FAKE)), v(k.get("g", FAKE)), k.get("token", 0),
        v(k.get("qg", FAKE)), k.get("dt", 1), k.get("pt", 0), f(k.get("scale", 1.0)), f(k.get("eps", 1e-6)),
        v(k.get("s", FAKE)), v(k.get("n", FAKE)), v(k.get("post", FAKE)), v(k.get("pre", FAKE)), k.get("T", 4),
        k.get("D", 8), None)
    assert fwd(T=0) == OK
    assert fwd(T=0, b=0, s=0) == OK
    for bad in (dict(T=-1), dict(D=0), dict(dt=3), dict(pt=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(b=0), dict(r=0), dict(s=0), dict(n=0),
                dict(pre=0), dict(post=0)):  # the last: a gamma without its norm
        assert fwd(**bad) == INVALID, bad
    assert fwd(T=1 << 31) == SHAPE
    assert fwd(D=(1 << 24) + 1) == SHAPE
    for bad in (dict(b=FAKE + 1), dict(dt=0, s=FAKE + 2), dict(qg=FAKE + 2), dict(g=FAKE + 2), dict(token=1, g=FAKE + 1),
                dict(pre=FAKE + 2)):
        assert fwd(**bad) == MISALIGNED, bad
    need = binding.moe_block_norm_bwd_workspace_bytes(4, 8)
    bwd = lambda **k: lib.moe_block_norm_bwd(
        v(k.get("ds", FAKE)), v(k.get("dn", FAKE)), v(k.get("b", FAKE)), v(k.get("s", FAKE)), v(k.get("pg", FAKE)),
        v(k.get("g", FAKE)), k.get("token", 0), v(FAKE), v(k.get("post", FAKE)), v(k.get("pre", FAKE)), k.get("dt", 2),
        k.get("pt", 2), f(k.get("scale", 1.0)), v(k.get("db", FAKE)), v(k.get("dr", FAKE)), v(k.get("dpg", FAKE)),
        v(k.get("dg", FAKE)), v(k.get("dqg", FAKE)), k.get("T", 4), k.get("D", 8), v(k.get("ws", FAKE)),
        k.get("wsb", need), None)
    for bad in (dict(T=-1), dict(D=-8), dict(dt=9), dict(scale=float("nan")), dict(dn=0), dict(s=0), dict(pre=0),
                dict(db=0), dict(dr=0), dict(ws=0), dict(post=0), dict(post=0, pg=0), dict(g=0), dict(b=0),
                dict(b=0, post=0, pg=0, dpg=0)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(D=(1 << 24) + 1) == SHAPE
    for bad in (dict(db=FAKE + 1), dict(dpg=FAKE + 1), dict(dg=FAKE + 1), dict(ws=FAKE + 16), dict(dt=0, token=1, g=FAKE + 2)):
        assert bwd(**bad) == MISALIGNED, bad
    assert bwd(wsb=need - 1) == WS_SMALL
    assert binding.moe_block_norm_bwd_workspace_bytes(0, 8) == 0
    assert binding.moe_block_norm_bwd_workspace_bytes(4, WRAP + 8) == 0


# ---------------------------------------------------------------------- the layer for a few tokens

def test_few_refusals(lib):
    def fwd(**k):
        a = dict(x=FAKE, ids=FAKE, scores=FAKE, sd=0, w13=FAKE, w2=FAKE, out=FAKE, T=4, D=128, F=64, E=8, K=2, ws=FAKE,
                 wsb=1 << 30)
        a.update(k)
        return lib.moe_routed_experts_fwd_few(
            v(a["x"]), v(a["ids"]), v(a["scores"]), a["sd"], v(a["w13"]), v(a["w2"]), v(a["out"]), a["T"], a["D"], a["F"],
            a["E"], a["K"], v(a["ws"]), a["wsb"], None)

    def layer(**k):
        a = dict(x=FAKE, z=FAKE, dt=0, w13=FAKE, w2=FAKE, ids=FAKE, scores=FAKE, out=FAKE, T=4, D=128, F=64, E=8, K=2,
                 ws=FAKE, wsb=1 << 30)
        a.update(k)
        return lib.moe_layer_fwd_few(
            v(a["x"]), v(a["z"]), a["dt"], 1, v(a["w13"]), v(a["w2"]), v(a["ids"]), v(a["scores"]), v(a["out"]), a["T"],
            a["D"], a["F"], a["E"], a["K"], v(a["ws"]), a["wsb"], None)

    need = binding.moe_few_workspace_bytes(4, 128, 64, 8, 2)
    assert need >= 256 + 2 * 8 * 64
    for call in (fwd, layer):
        assert call(T=0) == OK
        assert call(T=0, x=0, ids=0) == OK
        for bad in (dict(T=-1), dict(D=0), dict(F=-64), dict(E=0), dict(K=0), dict(x=0), dict(ids=0), dict(scores=0),
                    dict(w13=0), dict(w2=0), dict(out=0), dict(ws=0)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(T=33), dict(T=32, E=32, K=17), dict(D=96), dict(F=100), dict(E=4097), dict(E=4096, F=1 << 18)):
            assert call(**bad) == SHAPE, bad
        for bad in (dict(x=FAKE + 8), dict(w13=FAKE + 4), dict(w2=FAKE + 8), dict(out=FAKE + 2), dict(ids=FAKE + 4),
                    dict(scores=FAKE + 8), dict(ws=FAKE + 16)):
            assert call(**bad) == MISALIGNED, bad
        assert call(wsb=need - 1) == WS_SMALL
    assert fwd(sd=2) == INVALID
    assert layer(dt=2) == INVALID
    assert layer(K=9) == INVALID
    assert layer(z=0) == INVALID
    assert layer(z=FAKE + 2) == MISALIGNED
    for sizes in ((0, 128, 64, 8, 2), (33, 128, 64, 8, 2), (4, 100, 64, 8, 2), (4, WRAP + 128, 64, 8, 2)):
        assert binding.moe_few_workspace_bytes(*sizes) == 0


# ---------------------------------------------------------------------- the choice of the next token

def test_sample_refusals(lib):
    go = lambda **k: lib.moe_sample(
        v(k.get("z", FAKE)), k.get("dt", 1), v(k.get("u", FAKE)), v(k.get("tau", 0)), v(k.get("k", 0)), v(k.get("p", FAKE)),
        v(0), v(k.get("token", FAKE)), v(k.get("lp", 0)), k.get("T", 4), k.get("V", 100), None)
    assert go(T=0) == OK
    assert go(T=0, z=0) == OK
    for bad in (dict(T=-1), dict(V=0), dict(dt=3), dict(dt=-1), dict(z=0), dict(u=0), dict(token=0)):
        assert go(**bad) == INVALID, bad
    assert go(T=1 << 31) == SHAPE
    assert go(V=(1 << 24) + 1) == SHAPE
    for bad in (dict(z=FAKE + 1), dict(dt=0, z=FAKE + 2), dict(u=FAKE + 2), dict(tau=FAKE + 1), dict(k=FAKE + 2),
                dict(p=FAKE + 2), dict(token=FAKE + 2), dict(lp=FAKE + 1)):
        assert go(**bad) == MISALIGNED, bad


# ---------------------------------------------------------------------- the binding's own checks

def calls(T, D, F, E, K):
    """The calls with tensors of these sizes."""
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    x, row, ws, p = tensor(T, D), tensor(T, dtype=f32), tensor(1 << 20, dtype=u8), tensor(D)
    w13, w2 = tensor(E, 2, F, D), tensor(E, D, F)
    ids, scores, z = tensor(T, K, dtype=i32), tensor(T, K, dtype=f32), tensor(T, E)
    number = tensor(T, dtype=i32)
    return {
        "moe_block_norm_fwd": lambda **k: binding.moe_block_norm_fwd(x, x, p, p, p, x, x, row, row, **k),
        "moe_block_norm_bwd": lambda **k: binding.moe_block_norm_bwd(x, x, x, x, p, p, p, row, row, x, x, p, p, p, ws, **k),
        "moe_routed_experts_fwd_few": lambda **k: binding.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, x, ws, **k),
        "moe_layer_fwd_few": lambda **k: binding.moe_layer_fwd_few(x, z, w13, w2, ids, scores, x, ws, **k),
        "moe_sample": lambda **k: binding.moe_sample(z, row, number, row, row, number, row, row, **k),
    }


SMALL = dict(T=4, D=64, F=64, E=8, K=2)
NAMES = list(calls(**SMALL))


@pytest.fixture
def called(monkeypatch):
    """The names of the library's functions that are called; the tensors lie on cuda:1, the current device is `called.at`."""
    class Names(list):
        at = 1
    names = Names()
    monkeypatch.setattr(binding, "load", lambda: Library(names))
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: names.at, raising=False)
    return names


@pytest.mark.parametrize("name", NAMES)
def test_devices_and_streams(called, name):
    call = calls(**SMALL)[name]
    call()
    call(stream=Stream(1))
    assert called == [name, name]
    with pytest.raises(ValueError, match="stream"):
        call(stream=Stream(0))
    called.at = 0
    for kw in ({}, {"stream": Stream(0)}, {"stream": 0}):
        with pytest.raises(ValueError, match="current device"):
            call(**kw)
    assert called == [name, name]


@pytest.mark.parametrize("name,size", [("moe_block_norm_fwd", "D"), ("moe_block_norm_bwd", "D"),
                                       ("moe_routed_experts_fwd_few", "F"), ("moe_routed_experts_fwd_few", "K"),
                                       ("moe_layer_fwd_few", "E"), ("moe_layer_fwd_few", "D"), ("moe_sample", "E")])
def test_sizes_past_32_bits(called, name, size):
    with pytest.raises(ValueError, match="32"):
        calls(**{**SMALL, size: WRAP + SMALL[size]})[name]()
    assert not called


def test_shapes_that_do_not_belong_together(called):
    x, row, p, ws = tensor(4, 64), tensor(4, dtype=torch.float32), tensor(64), tensor(1 << 20, dtype=torch.uint8)
    ids, scores = tensor(4, 2, dtype=torch.int32), tensor(4, 2, dtype=torch.float32)
    w13, w2 = tensor(8, 2, 64, 64), tensor(8, 64, 64)
    few = binding.moe_routed_experts_fwd_few
    for bad in (lambda: few(x, ids, scores, tensor(8, 3, 64, 64), w2, x, ws), lambda: few(x, ids, scores, w13, tensor(8, 64, 128), x, ws),
                lambda: few(x, ids, tensor(4, 3, dtype=torch.float32), w13, w2, x, ws),
                lambda: few(x, tensor(5, 2, dtype=torch.int32), scores, w13, w2, x, ws),
                lambda: few(x, ids, scores, w13, w2, tensor(4, 128), ws),
                lambda: binding.moe_layer_fwd_few(x, tensor(4, 7), w13, w2, ids, scores, x, ws),
                lambda: binding.moe_block_norm_fwd(x, x, tensor(63), None, None, x, x, row, row),
                lambda: binding.moe_block_norm_fwd(x, x, None, tensor(4, 63), None, x, x, row, row),
                lambda: binding.moe_block_norm_fwd(x, x, None, tensor(63), None, x, x, row, row),
                lambda: binding.moe_block_norm_bwd(x, x, x, x, None, x, None, row, row, x, x, None, p, None, ws)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: few(x, ids, tensor(4, 2, dtype=torch.float64), w13, w2, x, ws),
                lambda: few(tensor(4, 64, dtype=torch.float16), ids, scores, w13, w2, x, ws),
                lambda: binding.moe_layer_fwd_few(x, tensor(4, 8, dtype=torch.float16), w13, w2, ids, scores, x, ws),
                lambda: binding.moe_block_norm_fwd(x, x, p, tensor(64, dtype=torch.float32), None, x, x, row, row)):
        with pytest.raises(TypeError):
            bad()
    assert not called
