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
