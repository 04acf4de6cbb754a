"""Trains a small mixture-of-experts language model with this package's operators, forward and backward.

One block and a head, in bf16 with fp32 sums inside the operators:

    h0 = embedding[tokens]
    n1 = layer_norm(h0);  logits = n1 router^T;  ids, scores = top_k(logits)
    h1 = h0 + routed_experts(n1, ids, scores)
    n2 = layer_norm(h1);  loss = cross_entropy(n2 head^T, next tokens)

or, given a teacher's top logits, the distillation loss. ``forward_backward`` is the step a training loop
makes: every operator writes into buffers kept from step to step, and nothing synchronises. The embedding's
gather, the router's projection, the additions and the update are plain torch.

    python examples/train_moe_lm.py --steps 100            # next-token loss
    python examples/train_moe_lm.py --steps 100 --distill  # from a teacher's top 8 logits
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from mixture_experts_routed_topk_gb300 import binding as moe  # noqa: E402


class MoeLm:
    def __init__(self, tokens=1024, hidden=256, ffn=256, experts=8, top_k=2, vocab=2048, teacher_k=8, seed=0,
                 device="cuda"):
        self.T, self.D, self.F, self.E, self.K, self.V = tokens, hidden, ffn, experts, top_k, vocab
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).to(device)

        D, F, E, V, T = hidden, ffn, experts, vocab, tokens
        self.params = {
            "embedding": normal(V, D, std=1.0),
            "gamma1": torch.ones(D, device=device), "beta1": torch.zeros(D, device=device),
            "router": normal(E, D, std=D ** -0.5),
            "w13": normal(E, 2, F, D, std=D ** -0.5), "w2": normal(E, D, F, std=F ** -0.5),
            "gamma2": torch.ones(D, device=device), "beta2": torch.zeros(D, device=device),
            "head": normal(V, D, std=D ** -0.5),
        }
        self.grads = {name: torch.empty_like(p) for name, p in self.params.items()}

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)

        f32 = torch.float32
        self.n1, self.n2, self.moe_out = buf(T, D), buf(T, D), buf(T, D)
        self.mean1, self.rstd1, self.mean2, self.rstd2 = (buf(T, dtype=f32) for _ in range(4))
        self.ids, self.scores = buf(T, top_k, dtype=torch.int32), buf(T, top_k, dtype=f32)
        self.loss, self.lse = buf(T, dtype=f32), buf(T, dtype=f32)
        self.dn2, self.dh1, self.dn1, self.dh0 = (buf(T, D) for _ in range(4))
        self.dscores, self.dlogits = buf(T, top_k, dtype=f32), buf(T, experts, dtype=f32)
        dims = (T, D, F, E, top_k)
        self.ws_fwd = moe.alloc_workspace(moe.moe_workspace_bytes(*dims), device)
        self.ws_bwd = moe.alloc_workspace(moe.moe_bwd_workspace_bytes(*dims), device)
        self.ws_norm = moe.alloc_workspace(moe.moe_layernorm_bwd_workspace_bytes(T, D), device)
        self.ws_head = moe.alloc_workspace(moe.moe_lm_workspace_bytes(T, D, V, max(1, teacher_k)), device)
        self.dloss = torch.full((T,), 1.0 / T, device=device)

    def forward_backward(self, tokens, targets=None, teacher=None, temperature: float = 1.0):
        """Fills self.grads and returns the per-token losses. targets [T] int32 (-100: no loss), or teacher =
        (ids [T,k] int32, logits [T,k] fp32)."""
        p, g = self.params, self.grads
        h0 = p["embedding"][tokens]
        moe.moe_layernorm_fwd(h0, p["gamma1"], p["beta1"], self.n1, self.mean1, self.rstd1)
        logits = (self.n1 @ p["router"].T).float()
        moe.moe_router_topk_fwd(logits, self.ids, self.scores)
        moe.moe_routed_experts_fwd(self.n1, self.ids, self.scores, p["w13"], p["w2"], self.moe_out, self.ws_fwd)
        h1 = h0 + self.moe_out
        moe.moe_layernorm_fwd(h1, p["gamma2"], p["beta2"], self.n2, self.mean2, self.rstd2)
        if teacher is None:
            moe.moe_lm_ce_fwd(self.n2, p["head"], targets, self.loss, self.lse, self.ws_head)
            moe.moe_lm_ce_bwd(self.n2, p["head"], targets, self.lse, self.dloss, self.dn2, g["head"], self.ws_head)
        else:
            moe.moe_lm_distill_fwd(self.n2, p["head"], *teacher, self.loss, self.lse, self.ws_head, temperature)
            moe.moe_lm_distill_bwd(self.n2, p["head"], *teacher, self.lse, self.dloss, self.dn2, g["head"],
                                   self.ws_head, temperature)
        moe.moe_layernorm_bwd(self.dn2, h1, p["gamma2"], self.mean2, self.rstd2, self.dh1, g["gamma2"], g["beta2"],
                              self.ws_norm)
        moe.moe_routed_experts_bwd(self.n1, self.ids, self.scores, p["w13"], p["w2"], self.dh1, self.dn1,
                                   self.dscores, g["w13"], g["w2"], self.ws_bwd)
        moe.moe_router_topk_bwd(logits, self.ids, self.dscores, self.dlogits)
        dlogits = self.dlogits.to(torch.bfloat16)
        g["router"].copy_(dlogits.T @ self.n1)
        dn1 = self.dn1 + dlogits @ p["router"]
        moe.moe_layernorm_bwd(dn1, h0, p["gamma1"], self.mean1, self.rstd1, self.dh0, g["gamma1"], g["beta1"],
                              self.ws_norm)
        g["embedding"].zero_().index_add_(0, tokens, self.dh1 + self.dh0)
        return self.loss

    def status(self) -> int:
        """The device status bits of the step's last call on each workspace (synchronises). The loss's forward and
        backward share one, so the forward's bits last only until the backward, which raises bad targets again."""
        return moe.moe_get_status(self.ws_fwd) | moe.moe_get_status(self.ws_bwd) | moe.moe_get_status(self.ws_head)


class Adam:
    """Adam on fp32 copies of the parameters."""

    def __init__(self, model: MoeLm, lr: float = 3e-3):
        self.model, self.lr, self.t = model, lr, 0
        self.master = {n: p.float() for n, p in model.params.items()}
        self.m = {n: torch.zeros_like(p) for n, p in self.master.items()}
        self.v = {n: torch.zeros_like(p) for n, p in self.master.items()}

    def step(self):
        self.t += 1
        for n, p in self.model.params.items():
            g = self.model.grads[n].float()
            self.m[n].lerp_(g, 0.1)
            self.v[n].lerp_(g.square(), 0.01)
            m, v = self.m[n] / (1 - 0.9 ** self.t), self.v[n] / (1 - 0.99 ** self.t)
            self.master[n] -= self.lr * m / (v.sqrt() + 1e-8)
            p.copy_(self.master[n])


def batch(T: int, V: int, seed: int, device="cuda"):
    """Tokens of a fixed random successor table, with one token in ten drawn anew: something to learn."""
    table = torch.randperm(V, generator=torch.Generator().manual_seed(1234))
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, V, (T,), generator=g)
    y = torch.where(torch.rand(T, generator=g) < 0.1, torch.randint(0, V, (T,), generator=g), table[x])
    return x.to(device), y.to(torch.int32).to(device)


def teacher_of(targets, V: int, k: int, seed: int):
    """A made-up teacher: the target's logit high, k - 1 other tokens' lower."""
    g = torch.Generator().manual_seed(seed)
    other = torch.randint(1, V, (targets.numel(), k - 1), generator=g).cumsum(1).to(targets.device) + targets[:, None]
    ids = torch.cat([targets[:, None], other % V], 1).int()
    logits = torch.cat([torch.full((targets.numel(), 1), 6.0), torch.randn(targets.numel(), k - 1, generator=g)], 1)
    return ids.contiguous(), logits.to(targets.device)


def train(steps: int = 100, distill: bool = False, log=None, **sizes) -> list[float]:
    """Mean losses of the steps."""
    model = MoeLm(**sizes)
    opt, losses = Adam(model), []
    for step in range(steps):
        tokens, targets = batch(model.T, model.V, step)
        if distill:
            loss = model.forward_backward(tokens, teacher=teacher_of(targets, model.V, 8, step), temperature=2.0)
        else:
            loss = model.forward_backward(tokens, targets)
        losses.append(float(loss.mean()))
        if model.status():  # before the next step's calls clear it
            raise RuntimeError(f"step {step}: device status {model.status():#x}")
        opt.step()
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--distill", action="store_true", help="distil from a teacher's top 8 logits")
    args = ap.parse_args()
    train(args.steps, args.distill, log=print)
