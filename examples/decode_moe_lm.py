"""Generates tokens with a small mixture-of-experts language model, one decoding step for a few users at a time.

A step is, in bf16 with fp32 sums inside the operators,

    stream = embedding[tokens];  normed = rms(stream) pre_gamma
    for each block:  stream += gate rms(experts(normed)) post_gamma;  normed = rms(stream) pre_gamma
    tokens = a choice from normed head^T

The experts take each block's router logits (``moe_layer_fwd_few``), the norms around a block are one call
(``moe_block_norm_fwd``), and so is the choice (``moe_sample``). The embedding's gather and the two projections are plain
torch. A step allocates nothing that it keeps and does not synchronise, so it is captured once and replayed.

    python examples/decode_moe_lm.py --tokens 64 --users 4 --temperature 0.8 --top-k 40 --top-p 0.95
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from mixture_experts_routed_topk_gb300 import binding as moe  # noqa: E402


class MoeDecoder:
    def __init__(self, users=4, hidden=512, ffn=256, experts=16, top_k=4, blocks=2, vocab=4096, seed=0, device="cuda"):
        self.T, self.D, self.F, self.E, self.K, self.V, self.L = users, hidden, ffn, experts, top_k, vocab, blocks
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(device)

        T, D, F, E, V = users, hidden, ffn, experts, vocab
        f32 = torch.float32
        self.embedding, self.head = normal(V, D), normal(V, D, std=2.0 * D ** -0.5)
        # one norm before each block and before the head, one after each block
        self.pre_gamma = [normal(D, std=0.1, mean=1.0, dtype=f32) for _ in range(blocks + 1)]
        self.blocks = [dict(router=normal(E, D, std=D ** -0.5), w13=normal(E, 2, F, D, std=D ** -0.5),
                            w2=normal(E, D, F, std=F ** -0.5), post_gamma=normal(D, std=0.1, mean=1.0, dtype=f32),
                            gate=normal(D, std=0.1, mean=0.5, dtype=f32)) for _ in range(blocks)]

        def buf(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.tokens = torch.zeros(T, dtype=torch.int32, device=device)
        self.uniform, self.logprob = buf(T, dtype=f32), buf(T, dtype=f32)
        self.stream, self.normed, self.out = buf(T, D), buf(T, D), buf(T, D)
        self.post_rstd, self.pre_rstd = buf(T, dtype=f32), buf(T, dtype=f32)
        self.ids, self.scores = buf(T, top_k, dtype=torch.int32), buf(T, top_k, dtype=f32)
        self.ws = moe.alloc_workspace(moe.moe_few_workspace_bytes(T, D, F, E, top_k), device)
        self.choice = dict(temperature=None, top_k=None, top_p=None, min_p=None)

    def choose_with(self, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
        """How tokens are chosen from here on, the same for all users."""
        full = lambda v, dt: torch.full((self.T,), v, dtype=dt, device=self.tokens.device)
        self.choice = dict(temperature=full(temperature, torch.float32), top_k=full(top_k, torch.int32),
                           top_p=full(top_p, torch.float32), min_p=full(min_p, torch.float32))

    def logits(self):
        """The next tokens' logits [T,V] for self.tokens."""
        h = self.embedding[self.tokens.long()]
        # the first norm: a sum of which only the block's side counts
        moe.moe_block_norm_fwd(h, h, None, None, self.pre_gamma[0], self.stream, self.normed, None, self.pre_rstd,
                               residual_scale=0.0)
        for b, pre_gamma in zip(self.blocks, self.pre_gamma[1:]):
            moe.moe_layer_fwd_few(self.normed, self.normed @ b["router"].T, b["w13"], b["w2"], self.ids, self.scores,
                                  self.out, self.ws)
            moe.moe_block_norm_fwd(self.out, self.stream, b["post_gamma"], b["gate"], pre_gamma, self.stream, self.normed,
                                   self.post_rstd, self.pre_rstd)
        return self.normed @ self.head.T

    def step(self):
        """self.tokens becomes the next tokens for the numbers in self.uniform. Returns the logits."""
        z = self.logits()
        moe.moe_sample(z, self.uniform, self.tokens, self.logprob, **self.choice)
        return z

    def generate(self, prompt, n: int, seed: int = 0):
        """n tokens for each user after the last of the prompt's [T], from a captured step: [T, n] on the host."""
        draw = torch.Generator(device=self.tokens.device).manual_seed(seed)
        self.uniform.zero_()
        self.step()  # the operators' first calls, before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        self.tokens.copy_(prompt)
        said = torch.empty(n, self.T, dtype=torch.int32, device=self.tokens.device)
        for i in range(n):
            self.uniform.uniform_(generator=draw)
            graph.replay()
            said[i] = self.tokens
        if moe.moe_get_status(self.ws):
            raise RuntimeError(f"device status {moe.moe_get_status(self.ws):#x}")
        return said.T.cpu()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--users", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-k", type=int, default=40)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--min-p", type=float, default=0.0)
    ap.add_argument("--seed", type=int, default=0)
    args = ap.parse_args()
    model = MoeDecoder(users=args.users)
    model.choose_with(args.temperature, args.top_k, args.top_p, args.min_p)
    for user, text in enumerate(model.generate(torch.arange(args.users), args.tokens, args.seed).tolist()):
        print(f"user {user}:", *text)
