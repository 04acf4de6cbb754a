"""The operators of a decoding step together, as the example runs them, against the same step in 64 bits; and the norms
around a block with the experts between them, forward and backward, against torch's autograd in 64 bits."""

import os
import sys

import pytest
import torch

import block_norm_ref as N
import serve_ops_ref as S

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def exact_logits(m, tokens):
    """The logits in 64 bits, with the values that the step itself rounds to bf16 left as they are."""
    h = m.embedding[tokens.long()].double()
    stream = h
    normed = N.fwd(h, h, None, None, m.pre_gamma[0], 0.0, 1e-6, False)[1]
    for b, pre_gamma in zip(m.blocks, m.pre_gamma[1:]):
        z = normed @ b["router"].double().T
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)
        scores, ids = torch.softmax(top[:, :m.K], 1), ids[:, :m.K]
        out = torch.zeros_like(stream)
        for t in range(m.T):
            for k in range(m.K):
                e = int(ids[t, k])
                hid = torch.nn.functional.silu(b["w13"][e, 0].double() @ normed[t]) * (b["w13"][e, 1].double() @ normed[t])
                out[t] += scores[t, k] * (b["w2"][e].double() @ hid)
        stream, normed = N.fwd(out, stream, b["post_gamma"], b["gate"], pre_gamma, 1.0, 1e-6, True)[:2]
    return normed @ m.head.double().T


@pytest.mark.parametrize("users,top_k,experts", [(1, 4, 16), (5, 16, 16), (17, 8, 8)])
def test_a_step_of_the_example(users, top_k, experts):
    """top_k = experts where users are many: rounding the router's logits then moves scores, but no choice."""
    from decode_moe_lm import MoeDecoder

    m = MoeDecoder(users=users, hidden=256, ffn=128, experts=experts, top_k=top_k, vocab=1000, seed=users)
    m.choose_with(0.9, 30, 0.9, 0.001)
    g = torch.Generator().manual_seed(users)
    tokens = torch.randint(0, 1000, (users,), generator=g).int()
    m.tokens.copy_(tokens)
    m.uniform.copy_(torch.rand(users, generator=g))
    want = exact_logits(m, tokens.cuda())
    z = m.step()
    # some ten roundings to bf16 on the way, each of half a step, that add up as independent ones do at worst by three
    assert float((z.double() - want).norm() / want.norm()) < 3 * 10 ** 0.5 * 2.0 ** -8
    for t in range(users):
        token, logprob, _ = S.sample_row(z[t], float(m.uniform[t]), float(torch.tensor(0.9)), 30, float(torch.tensor(0.9)),
                                         float(torch.tensor(0.001)))
        assert int(m.tokens[t]) == token and abs(float(m.logprob[t]) - logprob) < 1e-6


def test_the_example_generates_what_its_steps_choose():
    from decode_moe_lm import MoeDecoder

    m = MoeDecoder(users=3, vocab=500)
    m.choose_with(0.8, 40, 0.95)
    text = m.generate(torch.tensor([1, 2, 3]), 12, seed=5)
    assert text.shape == (3, 12) and bool(((text >= 0) & (text < 500)).all())
    assert torch.equal(text, m.generate(torch.tensor([1, 2, 3]), 12, seed=5))
    # the same without a graph
    draw = torch.Generator(device="cuda").manual_seed(5)
    m.tokens.copy_(torch.tensor([1, 2, 3]))
    for i in range(12):
        m.uniform.uniform_(generator=draw)
        m.step()
        assert torch.equal(m.tokens.cpu(), text[:, i])
    m.choose_with(temperature=0.0)
    m.tokens.copy_(torch.tensor([1, 2, 3]))
    z = m.step()
    assert torch.equal(m.tokens.long(), z.argmax(1))


def test_a_block_between_its_norms_forward_and_backward():
    """normed -> experts -> norm, gate and residual -> normed, and back, as a training step runs it."""
    from mixture_experts_routed_topk_gb300 import binding as B

    T, D, F, E, K = 96, 256, 128, 8, 2
    g = torch.Generator().manual_seed(0)
    randn = lambda *s, std=1.0, mean=0.0, dt=BF16: (torch.randn(*s, generator=g) * std + mean).to(dt).cuda()
    stream0, w13, w2 = randn(T, D), randn(E, 2, F, D, std=D ** -0.5), randn(E, D, F, std=F ** -0.5)
    gammas = [randn(D, std=0.1, mean=1.0, dt=F32) for _ in range(3)]  # before the block, after it, before the next
    gate = randn(D, std=0.2, mean=0.5, dt=F32)
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().cuda()
    scores = torch.softmax(torch.randn(T, K, generator=g), 1).cuda()
    dstream, dnormed = randn(T, D), randn(T, D)
    new = lambda: torch.empty(T, D, dtype=BF16, device="cuda")
    vec = lambda: torch.empty(T, device="cuda")
    # forward
    s0, n0, r0 = new(), new(), vec()
    B.moe_block_norm_fwd(stream0, stream0, None, None, gammas[0], s0, n0, None, r0, residual_scale=0.0)
    out = new()
    dims = (T, D, F, E, K)
    B.moe_routed_experts_fwd(n0, ids, scores, w13, w2, out, B.alloc_workspace(B.moe_workspace_bytes(*dims)))
    s1, n1, post, pre = new(), new(), vec(), vec()
    B.moe_block_norm_fwd(out, s0, gammas[1], gate, gammas[2], s1, n1, post, pre)
    # backward
    ws = B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(T, D))
    dout, ds0, dn0, dx = new(), new(), new(), new()
    dg = [torch.empty(D, device="cuda") for _ in range(4)]  # the gammas' and the gate's gradients
    B.moe_block_norm_bwd(dstream, dnormed, out, s1, gammas[1], gate, gammas[2], post, pre, dout, ds0, dg[1], dg[3], dg[2], ws)
    dsc, dw13, dw2 = torch.empty(T, K, device="cuda"), torch.empty_like(w13), torch.empty_like(w2)
    B.moe_routed_experts_bwd(n0, ids, scores, w13, w2, dout, dn0, dsc, dw13, dw2,
                             B.alloc_workspace(B.moe_bwd_workspace_bytes(*dims)))
    B.moe_block_norm_bwd(ds0, dn0, None, s0, None, None, gammas[0], None, r0, dx, new(), None, None, dg[0], ws)
    # the same in 64 bits
    leaves = [t.double().requires_grad_() for t in (stream0, *gammas, gate, w13, w2, scores)]
    x, g0, g1, g2, ga, a13, a2, sc = leaves
    rms = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)
    n = rms(x) * g0
    y = torch.zeros_like(x)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        h = torch.nn.functional.silu(n[t] @ a13[e, 0].T) * (n[t] @ a13[e, 1].T)
        y = y.index_add(0, t, sc[t, k][:, None] * (h @ a2[e].T))
    s = x + ga * (rms(y) * g1)
    want = torch.autograd.grad((s * dstream.double()).sum() + (rms(s) * g2 * dnormed.double()).sum(), leaves)
    for name, a, b in zip(("stream", "pre_gamma", "post_gamma", "next pre_gamma", "gate", "w13", "w2", "scores"),
                          (dx, dg[0], dg[1], dg[2], dg[3], dw13, dw2, dsc), want):
        err = float((a.double() - b).norm() / b.norm())
        # fewer than ten roundings to bf16 lie on any way from the inputs to a gradient
        assert err < 3 * 10 ** 0.5 * 2.0 ** -8, (name, err)
