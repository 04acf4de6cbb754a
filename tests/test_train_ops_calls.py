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


class Library:
    """A library that notes which of its functions are called."""

    def __init__(self, called):
        self.called = called

    def __getattr__(self, name):
        return lambda *a: self.called.append(name) or 0


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
    """Sets the current device, for tensors that lie on cuda:1, and returns the names of the library's functions that
    are called."""
    called = []
    monkeypatch.setattr(binding, "load", lambda: Library(called))
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


# ------------------------------------------------------------------- sizes that do not fit the C arguments

class Tensor(torch.Tensor):
    """A tensor of a size that this machine does not have the memory for."""
    size_, dtype_ = (1, 1), torch.bfloat16
    shape = property(lambda self: torch.Size(self.size_))
    dtype = property(lambda self: self.dtype_)
    is_cuda = property(lambda self: True)

    def dim(self):
        return len(self.size_)

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE

    def numel(self):
        n = 1
        for s in self.size_:
            n *= s
        return n


def tensor(*size, dtype=torch.bfloat16):
    t = torch.zeros(1).as_subclass(Tensor)
    t.size_, t.dtype_ = size, dtype
    return t


def sized_calls(T, D, V, E, K, k, ignore=-100):
    """The eight calls with tensors of these sizes: V x D weights, E experts with K choices, k teacher entries."""
    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    x, w, row, ws = tensor(T, D), tensor(V, D), tensor(T, dtype=f32), tensor(1 << 20, dtype=u8)
    z, ids, scores = tensor(T, E), tensor(T, K, dtype=i32), tensor(T, K, dtype=f32)
    t, ti, tl = tensor(T, dtype=i32), tensor(T, k, dtype=i32), tensor(T, k, dtype=f32)
    return {
        "moe_layernorm_fwd": lambda: binding.moe_layernorm_fwd(x, tensor(D), tensor(D), x, row, row),
        "moe_layernorm_bwd": lambda: binding.moe_layernorm_bwd(x, x, None, row, row, x, None, None, None),
        "moe_router_topk_fwd": lambda: binding.moe_router_topk_fwd(z, ids, scores),
        "moe_router_topk_bwd": lambda: binding.moe_router_topk_bwd(z, ids, scores, z),
        "moe_lm_ce_fwd": lambda: binding.moe_lm_ce_fwd(x, w, t, row, row, ws, ignore),
        "moe_lm_ce_bwd": lambda: binding.moe_lm_ce_bwd(x, w, t, row, row, x, w, ws, ignore),
        "moe_lm_distill_fwd": lambda: binding.moe_lm_distill_fwd(x, w, ti, tl, row, row, ws),
        "moe_lm_distill_bwd": lambda: binding.moe_lm_distill_bwd(x, w, ti, tl, row, row, x, w, ws),
    }


SMALL = dict(T=4, D=64, V=100, E=8, K=2, k=3)
WRAP = 1 << 32  # a size of WRAP + n passed as a 32-bit number is n


@pytest.fixture
def checked(monkeypatch):
    """The names of the library's functions that are called, with cuda:1 as the current device."""
    called = []
    monkeypatch.setattr(binding, "load", lambda: Library(called))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    return called


@pytest.mark.parametrize("name", CALLS)
def test_sizes_that_fit(checked, name):
    sized_calls(**SMALL)[name]()
    assert checked == [name]


@pytest.mark.parametrize("name,size", [
    ("moe_layernorm_fwd", "D"), ("moe_layernorm_bwd", "D"), ("moe_router_topk_fwd", "E"), ("moe_router_topk_bwd", "E"),
    ("moe_router_topk_fwd", "K"), ("moe_router_topk_bwd", "K"), ("moe_lm_ce_fwd", "D"), ("moe_lm_ce_bwd", "V"),
    ("moe_lm_distill_fwd", "V"), ("moe_lm_distill_fwd", "k"), ("moe_lm_distill_bwd", "D"), ("moe_lm_distill_bwd", "k")])
def test_sizes_past_32_bits(checked, name, size):
    with pytest.raises(ValueError, match="32"):
        sized_calls(**{**SMALL, size: WRAP + SMALL[size]})[name]()
    assert not checked


def test_workspaces_of_sizes_past_32_bits():
    assert binding.moe_layernorm_bwd_workspace_bytes(4, WRAP + 64) == 0
    for sizes in ((4, WRAP + 64, 100, 1), (4, 64, WRAP + 100, 1), (4, 64, 100, WRAP + 1)):
        assert binding.moe_lm_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("name", ["moe_lm_ce_fwd", "moe_lm_ce_bwd"])
@pytest.mark.parametrize("ignore", [1 << 31, -(1 << 31) - 1, 1 << 32, (1 << 40) + 7])
def test_an_ignore_index_past_32_bits(checked, name, ignore):
    with pytest.raises(ValueError, match="ignore_index"):
        sized_calls(**SMALL, ignore=ignore)[name]()
    assert not checked
