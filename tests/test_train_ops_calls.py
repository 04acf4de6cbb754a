"""Calls of the operators around the expert layer that have to be refused before anything is launched, without a
GPU."""

import ctypes

import pytest
import torch

from mixture_experts_routed_topk_gb300 import binding, build

OK, INVALID = 0, 1
FAKE = 1 << 20  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


# the square is a factor of the loss, and its reciprocal of the logits: both have to stay within fp32
@pytest.mark.parametrize("tau", [1e-39, 1e-30, 2.0 ** -61, 2.0 ** 61, 1e30, 3.0e38])
def test_temperatures_whose_square_leaves_fp32(lib, tau):
    p, f = ctypes.c_void_p(FAKE), ctypes.c_float(tau)
    ws = binding.moe_lm_workspace_bytes(4, 64, 10, 3)
    assert lib.moe_lm_distill_fwd(p, p, p, p, f, p, p, 0, 64, 10, 3, p, ws, None) == INVALID
    assert lib.moe_lm_distill_bwd(p, p, p, p, f, p, p, None, None, 4, 64, 10, 3, p, ws, None) == INVALID


@pytest.mark.parametrize("tau", [2.0 ** -60, 1e-3, 1.0, 1e4, 2.0 ** 60])
def test_temperatures_that_are_taken(lib, tau):
    p, f = ctypes.c_void_p(FAKE), ctypes.c_float(tau)
    ws = binding.moe_lm_workspace_bytes(4, 64, 10, 3)
    assert lib.moe_lm_distill_fwd(p, p, p, p, f, p, p, 0, 64, 10, 3, p, ws, None) == OK  # no rows
    assert lib.moe_lm_distill_bwd(p, p, p, p, f, p, p, None, None, 4, 64, 10, 3, p, ws, None) == OK  # nothing asked for


# ------------------------------------------------------------------------------- the device of a call

class Stream:
    def __init__(self, device_index):
        self.device_index, self.cuda_stream = device_index, 0


CALLS = {
    "moe_layernorm_fwd": lambda t, **k: binding.moe_layernorm_fwd(t, t, t, t, t, t, **k),
    "moe_layernorm_bwd": lambda t, **k: binding.moe_layernorm_bwd(t, t, t, t, t, t, t, t, t, **k),
    "moe_router_topk_fwd": lambda t, **k: binding.moe_router_topk_fwd(t, t, t, **k),
    "moe_router_topk_bwd": lambda t, **k: binding.moe_router_topk_bwd(t, t, t, t, **k),
    "moe_lm_ce_fwd": lambda t, **k: binding.moe_lm_ce_fwd(t, t, t, t, t, t, **k),
    "moe_lm_ce_bwd": lambda t, **k: binding.moe_lm_ce_bwd(t, t, t, t, t, t, t, t, **k),
    "moe_lm_distill_fwd": lambda t, **k: binding.moe_lm_distill_fwd(t, t, t, t, t, t, t, **k),
    "moe_lm_distill_bwd": lambda t, **k: binding.moe_lm_distill_bwd(t, t, t, t, t, t, t, t, t, **k),
}


@pytest.fixture
def launches(monkeypatch):
    """The binding over a library that notes which of its functions are called, for tensors that lie on cuda:1 while
    a test's current device is its return value's."""
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(binding, "load", lambda: Library())
    monkeypatch.setattr(binding, "_rows", lambda x, name, dtypes: (4, 8, 1, FAKE))
    monkeypatch.setattr(binding, "_operand", lambda *a: FAKE)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)

    def current(device):
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: device, raising=False)
        return called
    return current


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_another_device_than_the_current_one(launches, name):
    called, t = launches(0), torch.zeros(4, 8)
    for kw in ({}, {"stream": Stream(0)}, {"stream": Stream(1)}, {"stream": 0}):
        with pytest.raises(ValueError, match="current device"):
            CALLS[name](t, **kw)
    assert not called


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device(launches, name):
    called, t = launches(1), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](t, stream=Stream(0))
    assert not called
    CALLS[name](t, stream=Stream(1))
    CALLS[name](t)
    assert called == [name, name]
