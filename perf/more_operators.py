"""The operators of a decoding step of a mixture-of-experts language model, as measured cases.

A block of such a model takes its output through a norm and a gate into the residual stream and
normalises the stream for what follows (``moe_block_norm_*``, which a training step also runs
backward); a decoding step has a handful of tokens to take through the routed experts
(``moe_routed_experts_fwd_few``, or ``moe_layer_fwd_few`` from the router's logits on), and ends with
the choice of the next token of each row (``moe_sample``). Each case is one pass of one of these, on
one GPU.

``run`` computes a case in plain torch operations (``own`` false; in 32 bits, the choice of a token in
64, where a sum of many small probabilities decides), or through the package's entry points (``own``
true). ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
FEW_MOST_BYTES = 9e9


# ------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's next token through the medium layer's experts: the shortest call of a decoding step
        dict(name="few_1_medium", op="few", T=1, D=2048, F=1408, E=64, K=6, route="ids", scores="f32"),
        # one token through the decode workload's experts, from the router's logits on
        dict(name="few_1_decode", op="few", T=1, D=7168, F=2048, E=256, K=8, route="logits", logits="f32",
             normalize=True),
        # a batch of 32 users on the skewed layer's sizes: most experts have a token or two
        dict(name="few_32_skewed", op="few", T=32, D=4096, F=1536, E=128, K=8, route="ids", scores="bf16"),
        # 16 users on the decode workload's sizes, scores that are a softmax over all experts
        dict(name="few_16_decode", op="few", T=16, D=7168, F=2048, E=256, K=8, route="logits", logits="bf16",
             normalize=False),
        # between two blocks of a decoding step of 16 users
        dict(name="norm_fwd_decode", op="norm_fwd", T=16, D=7168, dtype="bf16", param="bf16", gate="channel",
             post=True, scale=1.0),
        # rows of an odd length with a gate of their own for each token, as a conditioned block has
        dict(name="norm_fwd_odd", op="norm_fwd", T=8191, D=1001, dtype="f16", param="f32", gate="token",
             post=True, scale=0.5),
        # a training step's forward at the large layer's tokens
        dict(name="norm_fwd_large", op="norm_fwd", T=16384, D=7168, dtype="bf16", param="f32", gate="channel",
             post=True, scale=1.0),
        # its backward at the medium layer's sizes, without a norm after the block: residual sum and norm alone
        dict(name="norm_bwd_medium", op="norm_bwd", T=4096, D=2048, dtype="bf16", param="bf16", gate="none",
             post=False, scale=1.0),
        # its backward at the large layer's tokens, with both norms and the gate's gradient
        dict(name="norm_bwd_large", op="norm_bwd", T=16384, D=7168, dtype="bf16", param="f32", gate="channel",
             post=True, scale=1.0),
        # one user's next token from 32-bit logits, with the filters a chat serves with
        dict(name="sample_1_chat", op="sample", T=1, V=32000, dtype="f32", temperature=0.8, top_k=50, top_p=0.9,
             min_p=0.0, masked=False),
        # a batch over a large vocabulary from bf16 logits, the nucleus alone
        dict(name="sample_64_nucleus", op="sample", T=64, V=131072, dtype="bf16", temperature=1.0, top_k=0,
             top_p=0.95, min_p=0.0, masked=False),
        # an odd vocabulary with a third of it masked by a grammar, and a floor on the probability
        dict(name="sample_17_grammar", op="sample", T=17, V=50257, dtype="f32", temperature=1.0, top_k=0, top_p=1.0,
             min_p=0.02, masked=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["few", "few", "norm_fwd", "norm_bwd", "sample"])
    if op == "few":
        E = _log_int(rng, 4, 256)
        case = dict(op=op, T=_log_int(rng, 1, 32), D=64 * _log_int(rng, 4, 112), F=64 * _log_int(rng, 4, 32), E=E,
                    K=rng.randint(1, min(E, 8)), route=rng.choice(["ids", "logits"]))
        if case["route"] == "ids":
            case.update(scores=rng.choice(["f32", "bf16"]))
        else:
            case.update(logits=rng.choice(["f32", "bf16"]), normalize=rng.random() < 0.5)
        if work(case)["bytes"] > FEW_MOST_BYTES:
            case["T"] = max(1, case["T"] // 3)
        return case
    if op == "sample":
        return dict(op=op, T=_log_int(rng, 1, 256), V=_log_int(rng, 1000, 131072), dtype=rng.choice(["f32", "bf16"]),
                    temperature=rng.choice([0.7, 1.0, 1.2]), top_k=rng.choice([0, 0, 20, 200]),
                    top_p=rng.choice([0.5, 0.9, 0.98, 1.0]), min_p=rng.choice([0.0, 0.0, 0.05]),
                    masked=rng.random() < 0.3)
    D = _log_int(rng, 64, 7168)
    if rng.random() < 0.5:
        D = (D // 8) * 8
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    return dict(op=op, T=_log_int(rng, 1, 16384), D=D, dtype=dtype, param=rng.choice([dtype, "f32"]),
                gate=rng.choice(["none", "channel", "token"]), post=rng.random() < 0.7, scale=rng.choice([1.0, 0.5]))


# ------------------------------------------------------------------------------------------ inputs

def _prepare_few(c, g):
    T, D, F, E, K = c["T"], c["D"], c["F"], c["E"], c["K"]
    st = dict(
        x=torch.randn(T, D, generator=g, device="cuda").bfloat16(),  # normalised rows
        w13=torch.randn(E, 2, F, D, generator=g, device="cuda", dtype=torch.bfloat16).mul_(D ** -0.5),
        w2=torch.randn(E, D, F, generator=g, device="cuda", dtype=torch.bfloat16).mul_(F ** -0.5))
    logits = torch.randn(T, E, generator=g, device="cuda")
    if c["route"] == "logits":
        st["logits"] = logits.to(DTYPES[c["logits"]])
    else:
        top, ids = torch.topk(logits, K, dim=1)
        st.update(ids=ids.int().contiguous(), scores=torch.softmax(top, 1).to(DTYPES[c["scores"]]))
    return st


def _prepare_norm(c, g):
    T, D, dt, pt = c["T"], c["D"], DTYPES[c["dtype"]], DTYPES[c["param"]]

    def rows():
        return torch.randn(T, D, generator=g, device="cuda") * torch.exp(
            0.5 * torch.randn(T, 1, generator=g, device="cuda"))

    st = dict(block=rows().to(dt), residual=(2.0 * rows()).to(dt), eps=1e-6,
              pre_gamma=(1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt), post_gamma=None, gate=None)
    if c["post"]:
        st["post_gamma"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt)
    if c["gate"] == "channel":
        st["gate"] = (0.5 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(pt)
    elif c["gate"] == "token":
        st["gate"] = (0.5 + 0.2 * torch.randn(T, D, generator=g, device="cuda")).to(dt)
    if c["op"] == "norm_bwd":
        # what the forward pass kept, and the gradients that come back
        b = st["block"].float()
        st["post_rstd"] = torch.rsqrt(b.square().mean(1) + st["eps"]) if c["post"] else None
        u = b * st["post_rstd"][:, None] * st["post_gamma"].float() if c["post"] else b
        a = c["scale"] * st["residual"].float() + (u if st["gate"] is None else u * st["gate"].float())
        st["pre_rstd"] = torch.rsqrt(a.square().mean(1) + st["eps"])
        st["stream"] = a.to(dt)
        del st["residual"], b, u, a
        st["dstream"] = torch.randn(T, D, generator=g, device="cuda").to(dt)
        st["dnormed"] = torch.randn(T, D, generator=g, device="cuda").to(dt)
    return st


def _prepare_sample(c, g):
    T, V, dt = c["T"], c["V"], DTYPES[c["dtype"]]
    # frequent tokens first, noise, and a context that leans towards a few tokens
    z = 2.0 * torch.randn(T, V, generator=g, device="cuda") - torch.log1p(torch.arange(V, device="cuda"))
    likely = torch.randint(0, V, (T, 8), generator=g, device="cuda")
    z.scatter_add_(1, likely, 8.0 * torch.rand(T, 8, generator=g, device="cuda"))
    z = z.to(dt)
    if c["masked"]:  # every other row by the type's lowest value, the rest by -inf
        gone = torch.rand(T, V, generator=g, device="cuda") < 1.0 / 3.0
        low = torch.where(torch.arange(T, device="cuda")[:, None] % 2 == 0, torch.finfo(dt).min, -math.inf).to(dt)
        z = torch.where(gone, low, z)
    st = dict(logits=z.contiguous(), uniform=torch.rand(T, generator=g, device="cuda"), top_k=None, top_p=None,
              min_p=None)
    # each request its own temperature; one in eight takes the likeliest token
    t = c["temperature"] * (0.8 + 0.4 * torch.rand(T, generator=g, device="cuda"))
    st["temperature"] = torch.where(torch.rand(T, generator=g, device="cuda") < 0.125, 0.0, t) if T > 1 else t
    if c["top_k"]:
        st["top_k"] = torch.full((T,), c["top_k"], dtype=torch.int32, device="cuda")
    if c["top_p"] < 1.0:
        st["top_p"] = torch.full((T,), c["top_p"], device="cuda")
    if c["min_p"] > 0.0:
        st["min_p"] = torch.full((T,), c["min_p"], device="cuda")
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"few": _prepare_few, "norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm, "sample": _prepare_sample}
    return dict(make[case["op"]](case, g), case=case)


# ------------------------------------------------------------------------------------- plain forms

def _plain_few(st):
    c = st["case"]
    T, D, F, K = c["T"], c["D"], c["F"], c["K"]
    out = {}
    if c["route"] == "logits":
        z = st["logits"].float()
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)  # equal logits: the lowest id first
        top, ids = top[:, :K], ids[:, :K]
        e = torch.exp(top - top[:, :1])
        scores = e / (e.sum(1, keepdim=True) if c["normalize"] else torch.exp(z - top[:, :1]).sum(1, keepdim=True))
        out = {"ids": ids.int(), "scores": scores}
    else:
        ids, scores = st["ids"], st["scores"].float()
    flat = ids.reshape(-1).long()
    x = st["x"].float().repeat_interleave(K, 0)[:, :, None]
    gu = torch.matmul(st["w13"][flat].float().view(T * K, 2 * F, D), x)[:, :, 0]
    gate, up = gu[:, :F], gu[:, F:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(st["w2"][flat].float(), h[:, :, None]).view(T, K, D)
    out["out"] = (y * scores[:, :, None]).sum(1).bfloat16()
    return out


def _plain_norm_fwd(st):
    c = st["case"]
    b = st["block"].float()
    out = {}
    if c["post"]:
        out["post_rstd"] = torch.rsqrt(b.square().mean(1) + st["eps"])
        b = b * out["post_rstd"][:, None] * st["post_gamma"].float()
    if st["gate"] is not None:
        b = b * st["gate"].float()
    a = c["scale"] * st["residual"].float() + b
    out["pre_rstd"] = torch.rsqrt(a.square().mean(1) + st["eps"])
    out["stream"] = a.to(st["block"].dtype)
    out["normed"] = (a * out["pre_rstd"][:, None] * st["pre_gamma"].float()).to(st["block"].dtype)
    return out


def _plain_norm_bwd(st):
    c = st["case"]
    dt, pt = st["block"].dtype, st["pre_gamma"].dtype
    dn = st["dnormed"].float()
    hat = st["stream"].float() * st["pre_rstd"][:, None]
    gn = dn * st["pre_gamma"].float()
    da = st["dstream"].float() + st["pre_rstd"][:, None] * (gn - hat * (gn * hat).mean(1, keepdim=True))
    out = {"dpre_gamma": (dn * hat).sum(0).to(pt), "dresidual": (c["scale"] * da).to(dt)}
    b = st["block"].float()
    bh = b * st["post_rstd"][:, None] if c["post"] else b
    u = bh * st["post_gamma"].float() if c["post"] else bh
    du = da if st["gate"] is None else da * st["gate"].float()
    if c["gate"] == "channel":
        out["dgate"] = (da * u).sum(0).to(pt)
    elif c["gate"] == "token":
        out["dgate"] = (da * u).to(dt)
    if c["post"]:
        out["dpost_gamma"] = (du * bh).sum(0).to(pt)
        gb = du * st["post_gamma"].float()
        du = st["post_rstd"][:, None] * (gb - bh * (gb * bh).mean(1, keepdim=True))
    out["dblock"] = du.to(dt)
    return out


def _plain_sample(st):
    z = st["logits"].double()
    s, order = torch.sort(z, dim=1, descending=True, stable=True)  # equal logits: the lowest token first
    tau = st["temperature"].double()[:, None]
    greedy = tau <= 0.0
    w = torch.exp((s - s[:, :1]) / torch.where(greedy, torch.ones_like(tau), tau))
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    keep = torch.where(greedy, rank < 1, rank >= 0)
    if st["top_k"] is not None:
        keep = keep & (rank < st["top_k"][:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    if st["top_p"] is not None:  # the shortest run of the likeliest tokens that has this share
        keep = keep & (w.cumsum(1) - w < st["top_p"].double()[:, None] * w.sum(1, keepdim=True))
    if st["min_p"] is not None:
        keep = keep & (w >= st["min_p"].double()[:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    c = torch.zeros_like(w).scatter(1, order, w).cumsum(1)  # in the order of the tokens' numbers
    token = (c <= st["uniform"].double()[:, None] * c[:, -1:]).sum(1, keepdim=True)
    p = torch.zeros_like(w).scatter(1, order, w).gather(1, token) / c[:, -1:]
    return {"token": token[:, 0].int(), "logprob": torch.log(p)[:, 0].float()}


# ------------------------------------------------------------------------------- the package's calls

def _kept(st, name, make):
    """A buffer that a program keeps from step to step: made at the first use."""
    key = "kept_" + name
    if key not in st:
        st[key] = make()
    return st[key]


def _own_few(st, B):
    c = st["case"]
    T, K = c["T"], c["K"]
    ws = _kept(st, "ws", lambda: B.alloc_workspace(B.moe_few_workspace_bytes(T, c["D"], c["F"], c["E"], K), "cuda"))
    out = _kept(st, "out", lambda: torch.empty_like(st["x"]))
    if c["route"] == "ids":
        B.moe_routed_experts_fwd_few(st["x"], st["ids"], st["scores"], st["w13"], st["w2"], out, ws)
        return {"out": out}
    ids = _kept(st, "ids", lambda: torch.empty(T, K, dtype=torch.int32, device="cuda"))
    scores = _kept(st, "scores", lambda: torch.empty(T, K, device="cuda"))
    B.moe_layer_fwd_few(st["x"], st["logits"], st["w13"], st["w2"], ids, scores, out, ws, normalize=c["normalize"])
    return {"ids": ids, "scores": scores, "out": out}


def _own_norm_fwd(st, B):
    c = st["case"]
    T = c["T"]
    stream = _kept(st, "stream", lambda: torch.empty_like(st["block"]))
    normed = _kept(st, "normed", lambda: torch.empty_like(st["block"]))
    pre = _kept(st, "pre_rstd", lambda: torch.empty(T, device="cuda"))
    post = _kept(st, "post_rstd", lambda: torch.empty(T, device="cuda")) if c["post"] else None
    B.moe_block_norm_fwd(st["block"], st["residual"], st["post_gamma"], st["gate"], st["pre_gamma"], stream, normed,
                         post, pre, residual_scale=c["scale"], eps=st["eps"])
    out = {"stream": stream, "normed": normed, "pre_rstd": pre}
    return dict(out, post_rstd=post) if c["post"] else out


def _own_norm_bwd(st, B):
    c = st["case"]
    ws = _kept(st, "ws", lambda: B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(c["T"], c["D"]), "cuda"))
    dblock = _kept(st, "dblock", lambda: torch.empty_like(st["block"]))
    dresidual = _kept(st, "dresidual", lambda: torch.empty_like(st["block"]))
    dpre = _kept(st, "dpre", lambda: torch.empty_like(st["pre_gamma"]))
    dpost = _kept(st, "dpost", lambda: torch.empty_like(st["post_gamma"])) if c["post"] else None
    dgate = _kept(st, "dgate", lambda: torch.empty_like(st["gate"])) if c["gate"] != "none" else None
    B.moe_block_norm_bwd(st["dstream"], st["dnormed"], st["block"], st["stream"], st["post_gamma"], st["gate"],
                         st["pre_gamma"], st["post_rstd"], st["pre_rstd"], dblock, dresidual, dpost, dgate, dpre, ws,
                         residual_scale=c["scale"])
    out = {"dblock": dblock, "dresidual": dresidual, "dpre_gamma": dpre}
    if c["post"]:
        out["dpost_gamma"] = dpost
    if dgate is not None:
        out["dgate"] = dgate
    return out


def _own_sample(st, B):
    T = st["case"]["T"]
    token = _kept(st, "token", lambda: torch.empty(T, dtype=torch.int32, device="cuda"))
    logprob = _kept(st, "logprob", lambda: torch.empty(T, device="cuda"))
    B.moe_sample(st["logits"], st["uniform"], token, logprob, temperature=st["temperature"], top_k=st["top_k"],
                 top_p=st["top_p"], min_p=st["min_p"])
    return {"token": token, "logprob": logprob}


_PLAIN = {"few": _plain_few, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "sample": _plain_sample}
_OWN = {"few": _own_few, "norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "sample": _own_sample}


def run(state):
    if own:
        from mixture_experts_routed_topk_gb300 import binding

        return _OWN[state["case"]["op"]](state, binding)
    return _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- work, exact values

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "few":
        D, F, E, K = c["D"], c["F"], c["E"], c["K"]
        touched = max(1, round(E * (1.0 - (1.0 - K / E) ** T))) if T > 1 else K  # K distinct experts for each token
        route = T * E * SIZE[c["logits"]] + 8 * T * K if c["route"] == "logits" else T * K * (4 + SIZE[c["scores"]])
        return {"bytes": 6 * touched * F * D + 4 * T * D + route, "flops": 6 * T * K * F * D}
    if c["op"] == "sample":
        given = 8 + sum(4 for name, off in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)) if c[name] != off)
        return {"bytes": T * (c["V"] * SIZE[c["dtype"]] + given + 8), "flops": 4 * T * c["V"]}
    D, n = c["D"], T * c["D"]
    s, ps = SIZE[c["dtype"]], SIZE[c["param"]]
    params = ps * D * (1 + c["post"] + (c["gate"] == "channel"))
    stats = 4 * T * (1 + c["post"])
    if c["op"] == "norm_fwd":
        return {"bytes": (4 + (c["gate"] == "token")) * n * s + params + stats, "flops": 10 * n}
    # without a norm or a gate the block's gradient is the sum's alone, and the block itself is not needed
    reads = 4 if c["post"] or c["gate"] != "none" else 3
    return {"bytes": (reads + 2 + 2 * (c["gate"] == "token")) * n * s + 2 * params + stats, "flops": 22 * n}


def _exact_few(st):
    c = st["case"]
    T, K = c["T"], c["K"]
    out = {}
    if c["route"] == "logits":
        z = st["logits"].double()
        ids = torch.argsort(z, dim=1, descending=True, stable=True)[:, :K]
        scores = torch.softmax(z.gather(1, ids), 1) if c["normalize"] else torch.softmax(z, 1).gather(1, ids)
        out = {"ids": None, "scores": scores}
    else:
        ids, scores = st["ids"].long(), st["scores"].double()
    y = torch.zeros(T, c["D"], dtype=torch.float64, device="cuda")
    for e in torch.unique(ids).tolist():  # expert by expert, with the tokens that chose it
        t, k = torch.nonzero(ids == e, as_tuple=True)
        x = st["x"][t].double()
        h = torch.nn.functional.silu(x @ st["w13"][e, 0].double().T) * (x @ st["w13"][e, 1].double().T)
        y.index_add_(0, t, scores[t, k][:, None] * (h @ st["w2"][e].double().T))
    return dict(out, out=y)


def _exact_norm(st):
    c = st["case"]

    def rms(v, gamma):
        r = 1.0 / torch.sqrt((v * v).sum(1) / v.shape[1] + st["eps"])
        return r, v * r[:, None] * gamma

    if c["op"] == "norm_fwd":
        b, out = st["block"].double(), {}
        if c["post"]:
            out["post_rstd"], b = rms(b, st["post_gamma"].double())
        a = c["scale"] * st["residual"].double() + (b if st["gate"] is None else b * st["gate"].double())
        out["pre_rstd"], out["normed"] = rms(a, st["pre_gamma"].double())
        return dict(out, stream=a)
    # the gradients that torch's autograd finds, through the statistics that the forward pass kept
    dn, ds = st["dnormed"].double(), st["dstream"].double()
    a = st["stream"].double().requires_grad_()
    gamma = st["pre_gamma"].double().requires_grad_()

    def normed(v, kept):  # v / rms(v), where kept = 1 / rms(v) is given
        return v * (kept[:, None] - kept[:, None] ** 3 * (v.detach() * (v - v.detach())).mean(1, keepdim=True))

    da, dgamma = torch.autograd.grad(normed(a, st["pre_rstd"].double()) * gamma, (a, gamma), dn)
    da = da + ds
    del a, dn, ds
    out = {"dpre_gamma": dgamma, "dresidual": c["scale"] * da}
    leaves = {"block": st["block"].double().requires_grad_()}
    u = leaves["block"]
    if c["post"]:
        leaves["post_gamma"] = st["post_gamma"].double().requires_grad_()
        u = normed(u, st["post_rstd"].double()) * leaves["post_gamma"]
    if st["gate"] is not None:
        leaves["gate"] = st["gate"].double().requires_grad_()
        u = u * leaves["gate"]
    got = torch.autograd.grad(u, tuple(leaves.values()), da)
    out.update({"d" + name: grad for name, grad in zip(leaves, got)})
    return out


def _exact_sample(st):
    """A row at a time: the kept tokens by their thresholds, the running sum by a search."""
    T = st["case"]["T"]
    logprob = torch.empty(T, dtype=torch.float64, device="cuda")
    for t in range(T):
        z, tau = st["logits"][t].double(), float(st["temperature"][t])
        if tau <= 0.0:
            logprob[t] = 0.0
            continue
        order = torch.argsort(z, descending=True, stable=True)
        if st["top_k"] is not None:
            order = order[:int(st["top_k"][t])]
        p = torch.softmax(z[order] / tau, 0)
        n = p.numel()
        if st["top_p"] is not None:
            n = int(torch.searchsorted(p.cumsum(0), float(st["top_p"][t]))) + 1
        kept = order[:n]
        if st["min_p"] is not None:
            kept = kept[p[:n] >= float(st["min_p"][t]) * p[0]]
        kept = torch.sort(kept)[0]
        logp = torch.log_softmax(z[kept] / tau, 0)
        at = int(torch.searchsorted(torch.exp(logp).cumsum(0), float(st["uniform"][t]), right=True))
        logprob[t] = logp[min(at, kept.numel() - 1)]
    return {"token": None, "logprob": logprob}


def exact(case, seed):
    st = prepare(case, seed)
    find = {"few": _exact_few, "norm_fwd": _exact_norm, "norm_bwd": _exact_norm, "sample": _exact_sample}
    with torch.enable_grad():
        out = find[case["op"]](st)
    return {k: None if v is None else v.detach() for k, v in out.items()}
