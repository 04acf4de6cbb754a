"""The operators that stand around the routed-expert layer in a training step, as measured cases.

A block of a mixture-of-experts language model normalises its tokens (layer norm), lets a router
choose K of E experts per token, runs the expert layer, and at the end of the model turns hidden rows
into a loss: softmax cross entropy over the vocabulary, or the divergence from a teacher of which only
its top logits were kept. Each case is one pass of one of these, forward or backward, on one GPU.

``run`` computes a case in plain torch operations in 32 bits (``own`` false), or through the package's
entry points (``own`` true). ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the norm before the experts of a decode step of 64 tokens: a call of a few microseconds
        dict(name="ln_fwd_decode", op="ln_fwd", T=64, D=7168, dtype="bf16", param="bf16"),
        # rows of an odd length, so that no row after the first starts on a vector boundary
        dict(name="ln_fwd_odd", op="ln_fwd", T=8191, D=1001, dtype="f16", param="f32"),
        # the norm's backward in a training step of the medium layer, with both parameter gradients
        dict(name="ln_bwd_medium", op="ln_bwd", T=4096, D=2048, dtype="bf16", param="bf16"),
        # the same at the large layer's tokens, with the parameters kept in 32 bits
        dict(name="ln_bwd_large", op="ln_bwd", T=16384, D=7168, dtype="bf16", param="f32"),
        # the large layer's router: K of E from 32-bit logits, scores that sum to 1
        dict(name="router_fwd_large", op="router_fwd", T=16384, E=256, K=8, dtype="f32", normalize=True),
        # the medium layer's router backward, scores that are a softmax over all experts, bf16 logits
        dict(name="router_bwd_medium", op="router_bwd", T=4096, E=64, K=6, dtype="bf16", normalize=False),
        # scoring a handful of continuations: the head's weights are read once for 16 rows
        dict(name="ce_fwd_few", op="ce_fwd", T=16, D=2048, V=32000),
        # the loss of a training step over an odd vocabulary, a tenth of the rows ignored
        dict(name="ce_fwd_odd_vocab", op="ce_fwd", T=4096, D=4096, V=50257),
        # the head's backward in a training step of the medium layer
        dict(name="ce_bwd_medium", op="ce_bwd", T=4096, D=2048, V=32000),
        # and with a large vocabulary, whose logits alone would be 2 GB in bf16
        dict(name="ce_bwd_large_vocab", op="ce_bwd", T=8192, D=4096, V=131072),
        # distillation's loss on a ragged batch, 32 teacher logits to a row, some rows with fewer or none
        dict(name="distill_fwd_ragged", op="distill_fwd", T=2039, D=2048, V=32000, K=32, temperature=2.0),
        # distillation's backward with 64 teacher logits to a row, over an odd vocabulary
        dict(name="distill_bwd_odd_vocab", op="distill_bwd", T=4096, D=4096, V=50257, K=64, temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "router_fwd", "router_bwd", "ce_fwd", "ce_bwd", "distill_fwd", "distill_bwd"])
    if op.startswith("ln"):
        D = _log_int(rng, 64, 7168)
        if rng.random() < 0.5:
            D = (D // 8) * 8
        dtype = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, T=_log_int(rng, 1, 16384), D=D, dtype=dtype, param=rng.choice([dtype, "f32"]))
    if op.startswith("router"):
        E = _log_int(rng, 4, 512)
        return dict(op=op, T=_log_int(rng, 1, 32768), E=E, K=rng.randint(1, min(E, 12)),
                    dtype=rng.choice(["f32", "bf16"]), normalize=rng.random() < 0.5)
    # hidden sizes are multiples of 64, as the expert layer's are
    case = dict(op=op, T=_log_int(rng, 1, 8192), D=64 * (2 * (_log_int(rng, 4, 64) // 2) - 1),
                V=_log_int(rng, 1000, 131072))
    if op.startswith("distill"):
        case.update(K=_log_int(rng, 1, 128), temperature=rng.choice([1.0, 2.0, 4.0]))
    return case


# ------------------------------------------------------------------------------------------ inputs

def _head_inputs(c, g):
    """Hidden rows and head weights. A row leans towards the weight row of its (first) target, as a
    trained model's does: targets get a few percent of the probability, and some most of it."""
    T, D, V = c["T"], c["D"], c["V"]
    w = torch.randn(V, D, generator=g, device="cuda").mul_(1.0 / math.sqrt(D)).bfloat16()
    u = torch.rand(T, generator=g, device="cuda")
    targets = torch.exp(u * math.log(V)).long().sub_(1).clamp_(0, V - 1)  # frequent tokens first
    lean = 10.0 * torch.rand(T, 1, generator=g, device="cuda")
    x = torch.randn(T, D, generator=g, device="cuda") + lean * w[targets].float()
    return x.bfloat16(), w, targets


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = c["op"], c["T"]
    st = {"case": c}
    if op.startswith("ln"):
        D, dt, pt = c["D"], DTYPES[c["dtype"]], DTYPES[c["param"]]
        scale = torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda"))
        x = (torch.randn(T, D, generator=g, device="cuda") * scale
             + 0.3 * torch.randn(T, 1, generator=g, device="cuda")).to(dt)
        st.update(x=x, gamma=(1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt), eps=1e-5)
        if op == "ln_fwd":
            st["beta"] = (0.1 * torch.randn(D, generator=g, device="cuda")).to(pt)
        else:
            x32 = x.float()
            mean = x32.mean(1)
            st.update(mean=mean, rstd=torch.rsqrt((x32 - mean[:, None]).square().mean(1) + st["eps"]),
                      dy=torch.randn(T, D, generator=g, device="cuda").to(dt))
    elif op.startswith("router"):
        E, K = c["E"], c["K"]
        logits = torch.randn(T, E, generator=g, device="cuda").to(DTYPES[c["dtype"]])
        st["logits"] = logits
        if op == "router_bwd":
            st["ids"] = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :K].int().contiguous()
            st["dscores"] = torch.randn(T, K, generator=g, device="cuda")
    else:
        x, w, targets = _head_inputs(c, g)
        st.update(x=x, w=w)
        V = c["V"]
        if op.startswith("ce"):
            skip = torch.rand(T, generator=g, device="cuda") < 0.1
            st["targets"] = torch.where(skip, IGNORE, targets).int()
        else:
            K = min(c["K"], V)
            gaps = torch.randint(1, max(2, V // K), (T, K), generator=g, device="cuda")
            ids = (targets[:, None] + gaps.cumsum(1) - gaps[:, :1]) % V  # distinct, the target first
            top = torch.randn(T, K, generator=g, device="cuda").mul_(2.0).sort(1, descending=True)[0]
            kept = torch.randint(K // 2, K + 1, (T, 1), generator=g, device="cuda")
            kept[torch.rand(T, generator=g, device="cuda") < 0.05] = 0
            gone = torch.arange(K, device="cuda")[None, :] >= kept
            st["teacher_ids"] = torch.where(gone, -1, ids).int().contiguous()
            st["teacher_logits"] = torch.where(gone, torch.finfo(torch.float32).min, 8.0 + top).contiguous()
        if op.endswith("bwd"):
            st["dloss"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
            z = x.float() @ w.float().T
            st["lse"] = torch.logsumexp(z.div_(c.get("temperature", 1.0)), 1)
    return st


# ------------------------------------------------------------------------------------- plain forms

def _plain_ln_fwd(st):
    x = st["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + st["eps"])
    y = xc * rstd[:, None] * st["gamma"].float() + st["beta"].float()
    return {"y": y.to(st["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(st):
    dy = st["dy"].float()
    rstd = st["rstd"][:, None]
    xhat = (st["x"].float() - st["mean"][:, None]) * rstd
    g = dy * st["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    pt = st["gamma"].dtype
    return {"dx": dx.to(st["x"].dtype), "dgamma": (dy * xhat).sum(0).to(pt), "dbeta": dy.sum(0).to(pt)}


def _plain_router_fwd(st):
    c = st["case"]
    z = st["logits"].float()
    top, ids = torch.sort(z, dim=1, descending=True, stable=True)  # equal logits: the lowest index first
    top, ids = top[:, :c["K"]], ids[:, :c["K"]]
    m = top[:, :1]
    e = torch.exp(top - m)
    total = e.sum(1, keepdim=True) if c["normalize"] else torch.exp(z - m).sum(1, keepdim=True)
    return {"ids": ids.int(), "scores": e / total}


def _plain_router_bwd(st):
    c = st["case"]
    z = st["logits"].float()
    ids = st["ids"].long()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    top = e.gather(1, ids)
    total = top.sum(1, keepdim=True) if c["normalize"] else e.sum(1, keepdim=True)
    dot = (top / total * st["dscores"]).sum(1, keepdim=True)
    if c["normalize"]:
        dz = torch.zeros_like(z).scatter(1, ids, top / total * (st["dscores"] - dot))
    else:
        dz = e / total * (torch.zeros_like(z).scatter(1, ids, st["dscores"]) - dot)
    return {"dlogits": dz.to(st["logits"].dtype)}


def _plain_ce_fwd(st):
    z = st["x"].float() @ st["w"].float().T
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    valid = st["targets"] >= 0
    zt = z.gather(1, st["targets"].clamp(min=0).long()[:, None])[:, 0]
    return {"loss": torch.where(valid, lse - zt, torch.zeros_like(lse)), "lse": lse}


def _plain_ce_bwd(st):
    x, w = st["x"].float(), st["w"].float()
    q = torch.exp(x @ w.T - st["lse"][:, None])
    valid = st["targets"] >= 0
    t = st["targets"].clamp(min=0).long()[:, None]
    q.scatter_add_(1, t, torch.full_like(st["lse"], -1.0)[:, None])
    q *= (st["dloss"] * valid)[:, None]
    return {"dx": (q @ w).to(st["x"].dtype), "dw": (q.T @ x).to(st["w"].dtype)}


def _teacher(st):
    """The teacher's probabilities over its kept entries at the temperature (0 elsewhere), and which rows have any."""
    valid = st["teacher_ids"] >= 0
    a = torch.where(valid, st["teacher_logits"] / st["case"]["temperature"], -torch.inf)
    has = valid.any(1)
    m = torch.where(has, a.amax(1), torch.zeros_like(a[:, 0]))
    e = torch.exp(a - m[:, None])
    total = torch.where(has, e.sum(1), torch.ones_like(m))
    logp = torch.where(valid, a - m[:, None] - torch.log(total)[:, None], torch.zeros_like(a))
    return e / total[:, None], logp, has


def _plain_distill_fwd(st):
    tau = st["case"]["temperature"]
    z = st["x"].float() @ st["w"].float().T / tau
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    p, logp, has = _teacher(st)
    zt = z.gather(1, st["teacher_ids"].clamp(min=0).long())
    kl = (p * (logp - (zt - lse[:, None]))).sum(1)
    return {"loss": torch.where(has, tau * tau * kl, torch.zeros_like(kl)), "lse": lse}


def _plain_distill_bwd(st):
    tau = st["case"]["temperature"]
    x, w = st["x"].float(), st["w"].float()
    q = torch.exp(x @ w.T / tau - st["lse"][:, None])
    p, _, has = _teacher(st)
    q.scatter_add_(1, st["teacher_ids"].clamp(min=0).long(), -p)
    q *= (tau * st["dloss"] * has)[:, None]
    return {"dx": (q @ w).to(st["x"].dtype), "dw": (q.T @ x).to(st["w"].dtype)}


# ------------------------------------------------------------------------------- the package's calls

def _kept(st, name, make):
    """A buffer that a training loop keeps from step to step: made at the first use."""
    if name not in st:
        st[name] = make()
    return st[name]


def _own(st):
    from mixture_experts_routed_topk_gb300 import binding as B

    c = st["case"]
    op, T = c["op"], c["T"]
    if op == "ln_fwd":
        y = _kept(st, "y", lambda: torch.empty_like(st["x"]))
        mean = _kept(st, "mean", lambda: torch.empty(T, device="cuda"))
        rstd = _kept(st, "rstd", lambda: torch.empty(T, device="cuda"))
        B.moe_layernorm_fwd(st["x"], st["gamma"], st["beta"], y, mean, rstd, st["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        ws = _kept(st, "ws", lambda: B.alloc_workspace(B.moe_layernorm_bwd_workspace_bytes(T, c["D"]), "cuda"))
        dx = _kept(st, "dx", lambda: torch.empty_like(st["x"]))
        dgamma = _kept(st, "dgamma", lambda: torch.empty_like(st["gamma"]))
        dbeta = _kept(st, "dbeta", lambda: torch.empty_like(st["gamma"]))
        B.moe_layernorm_bwd(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"], dx, dgamma, dbeta, ws)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "router_fwd":
        ids = _kept(st, "ids", lambda: torch.empty(T, c["K"], dtype=torch.int32, device="cuda"))
        scores = _kept(st, "scores", lambda: torch.empty(T, c["K"], device="cuda"))
        B.moe_router_topk_fwd(st["logits"], ids, scores, normalize=c["normalize"])
        return {"ids": ids, "scores": scores}
    if op == "router_bwd":
        dlogits = _kept(st, "dlogits", lambda: torch.empty_like(st["logits"]))
        B.moe_router_topk_bwd(st["logits"], st["ids"], st["dscores"], dlogits, normalize=c["normalize"])
        return {"dlogits": dlogits}
    K = c.get("K", 1)
    ws = _kept(st, "ws", lambda: B.alloc_workspace(B.moe_lm_workspace_bytes(T, c["D"], c["V"], K), "cuda"))
    if op.endswith("fwd"):
        loss = _kept(st, "loss", lambda: torch.empty(T, device="cuda"))
        lse = _kept(st, "lse", lambda: torch.empty(T, device="cuda"))
        if op == "ce_fwd":
            B.moe_lm_ce_fwd(st["x"], st["w"], st["targets"], loss, lse, ws, ignore_index=IGNORE)
        else:
            B.moe_lm_distill_fwd(st["x"], st["w"], st["teacher_ids"], st["teacher_logits"], loss, lse, ws,
                                 temperature=c["temperature"])
        return {"loss": loss, "lse": lse}
    dx = _kept(st, "dx", lambda: torch.empty_like(st["x"]))
    dw = _kept(st, "dw", lambda: torch.empty_like(st["w"]))
    if op == "ce_bwd":
        B.moe_lm_ce_bwd(st["x"], st["w"], st["targets"], st["lse"], st["dloss"], dx, dw, ws, ignore_index=IGNORE)
    else:
        B.moe_lm_distill_bwd(st["x"], st["w"], st["teacher_ids"], st["teacher_logits"], st["lse"], st["dloss"], dx, dw,
                             ws, temperature=c["temperature"])
    return {"dx": dx, "dw": dw}


_PLAIN = {
    "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd,
    "router_fwd": _plain_router_fwd, "router_bwd": _plain_router_bwd,
    "ce_fwd": _plain_ce_fwd, "ce_bwd": _plain_ce_bwd,
    "distill_fwd": _plain_distill_fwd, "distill_bwd": _plain_distill_bwd,
}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- work, exact values

def work(case):
    c = case
    op, T = c["op"], c["T"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "ln_fwd":
        n = T * c["D"]
        return {"bytes": 2 * n * size[c["dtype"]] + 2 * c["D"] * size[c["param"]] + 8 * T, "flops": 8 * n}
    if op == "ln_bwd":
        n = T * c["D"]
        return {"bytes": 3 * n * size[c["dtype"]] + 3 * c["D"] * size[c["param"]] + 8 * T, "flops": 14 * n}
    if op == "router_fwd":
        n = T * c["E"]
        return {"bytes": n * size[c["dtype"]] + 8 * T * c["K"], "flops": 4 * n}
    if op == "router_bwd":
        n = T * c["E"]
        reads = T * c["K"] if c["normalize"] else n  # the chosen logits, or all of them
        return {"bytes": (reads + n) * size[c["dtype"]] + 8 * T * c["K"], "flops": 5 * n}
    D, V = c["D"], c["V"]
    targets = 8 * T * c["K"] if op.startswith("distill") else 4 * T
    product = 2 * T * D * V
    if op.endswith("fwd"):
        return {"bytes": 2 * (T + V) * D + targets + 8 * T, "flops": product}
    # the logits are not kept: the backward pass has their product once more, and two for the gradients
    return {"bytes": 4 * (T + V) * D + targets + 8 * T, "flops": 3 * product}


def _exact_head(st):
    c = st["case"]
    tau = c.get("temperature", 1.0)
    x = st["x"].double().requires_grad_()
    w = st["w"].double().requires_grad_()
    z = (x @ w.T) / tau
    lse = torch.logsumexp(z, dim=1)
    if c["op"].startswith("ce"):
        t = st["targets"].long()
        ok = t != IGNORE
        loss = torch.where(ok, -torch.log_softmax(z, 1).gather(1, torch.where(ok, t, 0)[:, None])[:, 0], 0.0)
    else:
        ids = st["teacher_ids"].long()
        kept = ids != -1
        logits = st["teacher_logits"].double().masked_fill(~kept, -math.inf) / tau
        some = kept.any(1)
        p = torch.where(some[:, None], torch.softmax(logits, 1), 0.0).nan_to_num(0.0)
        student = torch.log_softmax(z, 1).gather(1, ids.clamp(min=0))
        loss = tau ** 2 * (torch.special.xlogy(p, p) - p * student).sum(1)
    if c["op"].endswith("fwd"):
        return {"loss": loss.detach(), "lse": lse.detach()}
    dx, dw = torch.autograd.grad((loss * st["dloss"].double()).sum(), (x, w))
    return {"dx": dx, "dw": dw}


def exact(case, seed):
    if work(case)["flops"] > 8e12:  # 64-bit products run at about 1 TFLOP/s
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("ln"):
        x = st["x"].double().requires_grad_()
        gamma = st["gamma"].double().requires_grad_()
        beta = (st["beta"].double() if op == "ln_fwd" else torch.zeros_like(gamma)).requires_grad_()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + st["eps"]) * gamma + beta
        if op == "ln_fwd":
            return {"y": y.detach(), "mean": mean.detach()[:, 0], "rstd": 1.0 / torch.sqrt(var.detach()[:, 0] + st["eps"])}
        dx, dgamma, dbeta = torch.autograd.grad(y, (x, gamma, beta), st["dy"].double())
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op.startswith("router"):
        z = st["logits"].double().requires_grad_()
        ids = st["ids"].long() if "ids" in st else torch.argsort(z.detach(), dim=1, descending=True, stable=True)[:, :case["K"]]
        if case["normalize"]:
            scores = torch.softmax(z.gather(1, ids), 1)
        else:
            scores = torch.softmax(z, 1).gather(1, ids)
        if op == "router_fwd":
            return {"ids": None, "scores": scores.detach()}
        return {"dlogits": torch.autograd.grad(scores, z, st["dscores"].double())[0]}
    return _exact_head(st)
