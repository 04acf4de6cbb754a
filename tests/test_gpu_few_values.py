"""The layer for a few tokens where its answer hangs on more than its sums: what the kernel just before wrote, and H
near the end of its type."""

import pytest
import torch

from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("route", ["ids", "scores", "router", "logits f32", "logits bf16"])
def test_each_call_plans_from_what_was_just_written(route):
    """One pair and F = 64 give the gate/up kernel eight blocks, so the down kernel's 304 make their plans mostly on SMs
    where nothing has waited. A plan from the call before would take another expert's weights, or another score."""
    E, D, F, calls = 64, 7168, 64, 200
    g = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(1, D, generator=g, device="cuda").to(BF16)
    w13 = (torch.randn(E, 2, F, D, generator=g, device="cuda") * D ** -0.5).to(BF16)
    w2 = (torch.randn(E, D, F, generator=g, device="cuda") * F ** -0.5).to(BF16)
    ws = B.alloc_workspace(B.moe_few_workspace_bytes(1, D, F, E, 1))
    order = torch.randint(0, E, (calls,), generator=g, device="cuda")
    weight = 1.0 + torch.arange(calls, device="cuda") % 7 if route == "scores" else torch.ones(calls, device="cuda")
    logits_dtype = BF16 if route == "logits bf16" else F32
    logits = torch.nn.functional.one_hot(order, E).to(logits_dtype)  # each row's choice is order's, its score 1
    ids, scores = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    z, outs = torch.zeros(1, E, dtype=logits_dtype, device="cuda"), torch.zeros(calls, 1, D, dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    for i in range(calls):
        if route in ("ids", "scores"):
            ids.copy_(order[i:i + 1, None])
            scores.copy_(weight[i:i + 1, None])
            B.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, outs[i], ws)
        elif route == "router":
            B.moe_router_topk_fwd(logits[i:i + 1], ids, scores)
            B.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, outs[i], ws)
        else:
            z.copy_(logits[i:i + 1])
            B.moe_layer_fwd_few(x, z, w13, w2, ids, scores, outs[i], ws)
    torch.cuda.synchronize()
    want = {}
    for i in range(calls):
        key = int(order[i]), float(weight[i])
        if key not in want:  # inputs of its own that nothing writes again
            one = torch.full((1, 1), key[0], dtype=torch.int32, device="cuda"), torch.full((1, 1), key[1], device="cuda")
            torch.cuda.synchronize()
            want[key] = torch.empty_like(x)
            B.moe_routed_experts_fwd_few(x, *one, w13, w2, want[key], ws)
            torch.cuda.synchronize()
        assert torch.equal(outs[i], want[key]), i


@pytest.mark.parametrize("tokens", [1, 9, 20])
def test_h_near_the_end_of_bf16(tokens):
    """H = g u past bf16's largest number and within fp32's stays finite, beyond fp32's it is infinite; not a number it
    is only where a formula in any number of bits says so."""
    D, F = 128, 64
    x = torch.ones(tokens, D, dtype=BF16, device="cuda")
    w13, w2 = torch.zeros(5, 2, F, D, dtype=BF16, device="cuda"), torch.zeros(5, D, F, dtype=BF16, device="cuda")
    at = 11
    # g = SiLU(g) = 2^64 (1 - 2^-k) in two products, u = 2^64 or -2^64, H = 2^128 (1 - 2^-k)
    for e, (k, sign) in enumerate([(9, 1.0), (12, -1.0), (20, 1.0)]):
        w13[e, 0, at, 3], w13[e, 0, at, 70], w13[e, 1, at, 5] = 2.0 ** 64, -2.0 ** (64 - k), sign * 2.0 ** 64
    w13[3, 0, at, 3], w13[3, 1, at, 5] = 2.0 ** 64, 2.0 ** 64  # 2^128
    w13[4, 0, at, 3], w13[4, 1, at, 5] = 2.0 ** 64, -2.0 ** 64
    w2[:, :, at] = 2.0 ** -100
    want = [2.0 ** 28 * (1 - 2.0 ** -9), -2.0 ** 28 * (1 - 2.0 ** -12), 2.0 ** 28 * (1 - 2.0 ** -20), float("inf"),
            float("-inf")]
    ws = B.alloc_workspace(B.moe_few_workspace_bytes(tokens, D, F, 5, 1))
    for e, value in enumerate(want):
        out = torch.full_like(x, 7.0)
        B.moe_routed_experts_fwd_few(x, torch.full((tokens, 1), e, dtype=torch.int32, device="cuda"),
                                     torch.ones(tokens, 1, device="cuda"), w13, w2, out, ws)
        got = out.double()
        assert torch.equal(got, torch.full_like(got, got[0, 0])) and (float(got[0, 0]) == value or
                                                                      abs(float(got[0, 0]) - value) <= 2.0 ** -8 * abs(value)), e
