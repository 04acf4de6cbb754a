"""The weights behind the choice of the next token, where the tokens of ordinary rows say little about them: each weight
from the logarithm of a probability near 1, tokens with a border next to their number, vocabularies whose rare tokens
only count together, ties under a floor that nothing but the largest passes."""

import math

import pytest
import torch

import serve_ops_ref as S
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# A weight exp((z - max) / tau) is 2^(k/256) times 1 + f with f = x + x^2/2 + x^3/6 and 0 <= x < ln 2 / 256 = 2.8e-3, up
# to a rounding of x's argument. In steps of 2^-24 relative to f: the argument's sum has half a unit below 1 (8e-11 of the
# weight), the constant and the product one step each (3.2e-10), the polynomial's last sum and the product one each
# (3.2e-10), f in units of 2^-32 half a unit (1.2e-10); the next term x^4/24 is 2e-12. Together 8.4e-10 < 2^-30.
WEIGHT = 2.0 ** -30
UNIT = 2.0 ** -44  # whole units, cut off


def sample(z, u, **kw):
    T = z.shape[0]
    token, logprob = torch.full((T,), -7, dtype=torch.int32, device="cuda"), torch.full((T,), 7.0, device="cuda")
    vec = {k: torch.full((T,), v, dtype=torch.int32 if k == "top_k" else F32, device="cuda") for k, v in kw.items()}
    B.moe_sample(z.cuda(), torch.as_tensor(u, dtype=F32).expand(T).contiguous().cuda(), token, logprob, **vec)
    return token.cpu(), logprob.cpu().double()


@pytest.mark.parametrize("tau", [1.0, 0.7, 1.9])
@pytest.mark.parametrize("top", [0.0, 13.7, -250.125])
def test_each_weight(top, tau):
    """The likelier of two tokens has the probability 1 / (1 + w), whose logarithm is -w (1 - w / 2 + ..): an fp32 number
    near 0 that shows the weight to 2^-24 of itself."""
    g = torch.Generator().manual_seed(int(10 * tau))
    z = torch.empty(40000, 2)
    z[:, 0] = top
    z[:, 1] = z[:, 0] - (1.0 + 16.0 * torch.rand(40000, generator=g))
    token, logprob = sample(z, 0.0, temperature=tau)
    assert not token.any()
    tau = float(torch.tensor(tau, dtype=F32))
    w = torch.exp((z[:, 1].double() - z[:, 0].double()) / tau)
    want = -torch.log1p(w)
    bound = w * WEIGHT + UNIT + 2.0 ** -24 * want.abs() + 2.0 ** -52
    off = (logprob - want).abs() / bound
    assert float(off.max()) <= 1.0, (float(off.max()), z[off.argmax()].tolist())


@pytest.mark.parametrize("tau", [1.0, 1.3])
def test_numbers_next_to_a_border(tau):
    """Two tokens whose border lies 1e-9 to 8e-9 from an fp32 number: on its right side with weights good to 2^-30."""
    g = torch.Generator().manual_seed(7)
    z = torch.zeros(1 << 19, 2)
    z[:, 1] = -0.5 - 9.0 * torch.rand(1 << 19, generator=g)
    t = float(torch.tensor(tau, dtype=F32))
    border = 1.0 / (1.0 + torch.exp(z[:, 1].double() / t))
    u = border.to(F32)
    off = u.double() - border
    near = (off.abs() >= 1e-9) & (off.abs() <= 8e-9)
    z, u, off = z[near], u[near], off[near]
    assert z.shape[0] > 2000
    token, _ = sample(z, u, temperature=tau)
    assert torch.equal(token, (off > 0).int())


def flat_row(V, weight, jitter=0.0, dtype=F32, seed=0):
    """A row with one logit of 0 at a third of it, the others near log(weight)."""
    g = torch.Generator(device="cuda").manual_seed(V + seed)
    z = math.log(weight) - jitter * torch.rand(1, V, generator=g, device="cuda")
    z[0, V // 3] = 0.0
    return z.to(dtype)


def running(z, keep=None):
    """The running sums of the kept weights by number, in 64 bits, relative to the largest."""
    w = torch.exp(z[0].double() - z[0].double().max())
    w = w if keep is None else torch.where(keep, w, 0.0)
    return w.cumsum(0)


def lost(V):
    """What V tokens lose by whole units, as a share of the weights: less than a unit each, of 2^-44 of the largest below
    V = 2^19, and from there on of one in which the row's sum is 2^61 or so."""
    return V * (UNIT if V < 1 << 19 else 2.0 ** -61)


# vocabularies around the one from which V weights of 2^44 units take 63 bits; and weights just below the unit in which
# all V could be the largest and stay below 2^62, near it, and well above
SIZES = [200000, 262144, (1 << 19) - 1, 1 << 19, 600001, 1 << 20, (1 << 22) + 5, 1 << 24]


@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("octaves", [-0.01, 0.9, 3.3, 12.0])
def test_rare_tokens_count_together(V, octaves):
    weight = 2.0 ** (octaves - (62 - V.bit_length() + (V & (V - 1) == 0)))
    for jitter in (0.0, 0.7):
        z = flat_row(V, weight, jitter)
        run = running(z)
        S_all, top = float(run[-1]), V // 3
        bound = WEIGHT + lost(V)
        # the likeliest token's probability
        head = float(run[top - 1] / run[-1])
        numbers = [head + 0.5 / S_all] + [i / 8 for i in range(8)] + [1 - 2.0 ** -i for i in (12, 16, 20, 23, 24)]
        numbers += [head * i / 5 for i in range(5)]
        u = torch.tensor(numbers, dtype=F32)
        token, logprob = sample(z.expand(len(numbers), V).contiguous(), u)
        share = (run / run[-1]).cpu()
        for i, t in enumerate(token.tolist()):
            lo, hi = float(share[t - 1]) if t else 0.0, float(share[t])
            assert lo - bound <= float(u[i]) <= hi + bound, (i, t, lo, hi, float(u[i]))
            want = float(z[0, t]) - math.log(S_all)
            # a rare token's own weight is good to a unit of its own
            assert abs(float(logprob[i]) - want) <= 2.0 ** -24 * abs(want) + 2.0 * bound, (i, t, float(logprob[i]), want)


@pytest.mark.parametrize("V", [262144, 1 << 19, 1 << 20, 1 << 24])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_nucleus_that_ends_among_rare_tokens(V, dtype):
    weight = 2.0 ** (0.4 - (62 - V.bit_length() + 1))
    z = flat_row(V, weight, 0.5, dtype)
    w = torch.sort(torch.exp(z[0].double()), descending=True)[0].cumsum(0)
    S_all = float(w[-1])
    for part in (0.25, 0.6):  # of the rare tokens' weight
        p = float(torch.tensor((1.0 + part * (S_all - 1.0)) / S_all, dtype=F32))
        token, logprob = sample(z, (float(running(z)[V // 3 - 1]) + 0.5) / S_all, top_p=p)
        assert int(token[0]) == V // 3
        kept = math.exp(-float(logprob[0]))  # the kept weights' sum
        n = int((w < p * S_all).sum()) if p < 1.0 else V - 1  # a share that rounds to 1 keeps all
        bound = 4 * (WEIGHT + lost(V)) + 2.0 ** -24 * (S_all - 1.0)
        assert float(w[n - 1]) - bound <= kept <= float(w[min(n + 1, V - 1)]) + bound


@pytest.mark.parametrize("T,V", [(3, 262144), (2, 524287), (40, 530000), (200, 524288)])
@pytest.mark.parametrize("kw", [{}, dict(temperature=1.4), dict(top_k=60), dict(top_p=0.9), dict(min_p=0.02),
                                dict(top_k=5000, top_p=0.97), dict(temperature=math.inf)])
def test_large_vocabularies(T, V, kw):
    """Rows of ordinary logits, and of equal ones: every number of blocks to a row."""
    g = torch.Generator().manual_seed(T)
    z = torch.randn(T, V, generator=g) * 2.0 - torch.log1p(torch.arange(V))
    z[0] = 0.25
    z, u = z.cuda(), torch.rand(T, generator=g)
    token, _ = sample(z, u, **kw)
    sure = 0
    for t in range(min(T, 12)):
        want, _, near = S.sample_row(z[t], float(u[t]), kw.get("temperature", 1.0), kw.get("top_k", 0),
                                     float(torch.tensor(kw.get("top_p", 1.0))), float(torch.tensor(kw.get("min_p", 0.0))))
        if near >= WEIGHT + lost(V):
            sure += 1
            assert int(token[t]) == want, t
    assert sure >= min(T, 12) - 2


@pytest.mark.parametrize("least", [1.0, 1.5, math.inf])
@pytest.mark.parametrize("V", [50, 5000, 70000])
@pytest.mark.parametrize("tau", [1.0, math.inf])
def test_floors_that_only_the_largest_passes(V, tau, least):
    """w >= min_p keeps the tokens that tie for the largest logit at 1, and above 1 only the first of the order."""
    g = torch.Generator().manual_seed(V)
    z = torch.randn(16, V, generator=g)
    ties = torch.stack([torch.randperm(V, generator=g)[:5] for _ in range(16)])
    z.scatter_(1, ties, 9.0)
    z[1, ties[1]] = math.inf
    token, logprob = sample(z, torch.arange(16) / 16.0, temperature=tau, min_p=least)
    for t in range(16):
        order = sorted(ties[t].tolist())
        if least > 1.0:
            assert int(token[t]) == order[0] and float(logprob[t]) == 0.0, t
        elif tau == 1.0:
            assert int(token[t]) == order[int(5 * t / 16)] and abs(float(logprob[t]) + math.log(5)) < 1e-6, t
