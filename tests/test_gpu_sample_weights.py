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
