"""The choice of the next token on the GPU against the 64-bit one, token for token: every number of blocks to a row,
types, vocabularies that are no multiple of anything, filters alone and together, ties, masked tokens and rows."""

import math

import pytest
import torch

import serve_ops_ref as S
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# A number this near to a border may fall to either side: weights are good to 2^-32 of themselves, the table and the
# rounding of the temperature's reciprocal to as much.
NEAR = 2.0 ** -30


def make(T, V, dtype, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(1000 * seed + 31 * T + V)
    z = (torch.randn(T, V, generator=g) * scale - torch.log1p(torch.arange(V))).to(dtype)
    return z, torch.rand(T, generator=g)


def run(z, u, tau=None, k=None, p=None, least=None, stream=None):
    T = z.shape[0]
    vec = lambda x, dt: None if x is None else torch.as_tensor(x, dtype=dt).expand(T).contiguous().cuda()
    token, logprob = torch.full((T,), -7, dtype=torch.int32, device="cuda"), torch.full((T,), 7.0, device="cuda")
    B.moe_sample(z.cuda(), u.cuda(), token, logprob, vec(tau, F32), vec(k, torch.int32), vec(p, F32), vec(least, F32),
                 stream=stream)
    return token.cpu(), logprob.cpu()


def compare(z, u, tau=None, k=None, p=None, least=None):
    token, logprob = run(z, u, tau, k, p, least)
    pick = lambda x, t, other: other if x is None else float(torch.as_tensor(x, dtype=F32).expand(z.shape[0])[t])
    sure = 0
    for t in range(z.shape[0]):
        want, logp, near = S.sample_row(z[t], float(u[t]), pick(tau, t, 1.0), int(pick(k, t, 0)), pick(p, t, 1.0),
                                        pick(least, t, 0.0))
        if near < NEAR:
            continue
        sure += 1
        assert int(token[t]) == want, (t, int(token[t]), want, near)
        got = float(logprob[t])
        if math.isnan(logp):
            assert math.isnan(got)
        else:  # one rounding to fp32, and weights good to 2^-32
            assert abs(got - logp) <= 2.0 ** -24 * abs(logp) + 2.0 ** -30, (t, got, logp)
    assert sure >= z.shape[0] - 1 - z.shape[0] // 50
    return token


FILTERS = {
    "plain": {}, "warm": dict(tau=1.7), "k": dict(tau=0.8, k=40), "p": dict(p=0.9), "least": dict(least=0.03),
    "all": dict(tau=0.9, k=300, p=0.95, least=0.001), "wide": dict(tau=1.3, p=0.9995), "large k": dict(k=777),
    "one": dict(p=0.0), "k one": dict(k=1), "off": dict(k=0, p=1.0, least=0.0),
}


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", FILTERS)
@pytest.mark.parametrize("T,V", [(7, 1), (5, 3), (6, 1000), (40, 4099), (3, 32000), (1, 50257), (2, 131072)])
def test_tokens(T, V, dtype, name):
    compare(*make(T, V, dtype), **FILTERS[name])


@pytest.mark.parametrize("T", [1, 20, 60, 100, 200, 700])
def test_every_number_of_blocks_to_a_row(T):
    z, u = make(T, 16400, BF16, seed=1)
    compare(z, u, k=50, p=0.9)
    compare(z, u)


def test_each_row_has_its_own():
    z, u = make(64, 5000, F32, seed=2)
    i = torch.arange(64)
    compare(z, u, tau=torch.where(i % 5 == 0, 0.0, 0.3 + 0.05 * i), k=torch.where(i % 3 == 0, 0, i), p=0.3 + i / 64.0,
            least=torch.where(i % 2 == 0, 0.0, i / 640.0))


@pytest.mark.parametrize("u", [0.0, 2.0 ** -149, 2.0 ** -30, 0.5, 1.0 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan, math.inf])
def test_numbers_at_the_ends(u):
    z, _ = make(4, 3000, F32, seed=3)
    token, _ = run(z, torch.full((4,), u), k=50)
    for t in range(4):
        assert int(token[t]) == S.sample_row(z[t], 1.0 if u == math.inf else u, k=50)[0]


@pytest.mark.parametrize("tau", [0.0, -1.0, math.nan, 2.0 ** -61, 1e-12, 1e-3, 50.0, 1e30, math.inf])
def test_temperatures(tau):
    z, u = make(9, 4000, F32, seed=4)
    z[3, 17:40] = z[3].max() + 1.0  # several largest
    if tau == math.inf:  # all alike
        token, logprob = run(z, u, tau=tau)
        assert torch.equal(token, (u.double() * 4000).floor().int())
        assert torch.allclose(logprob, torch.full((9,), -math.log(4000.0)))
        token, _ = run(z, u, tau=tau, k=23)
        assert bool(((token >= 17) & (token < 40))[3])
    else:
        compare(z, u, tau=tau)
        compare(z, u, tau=tau, k=30, p=0.8)


def test_minimum_shares():
    z, u = make(8, 3000, F32, seed=5)
    for least in (1.0, 2.0, 0.999, 1e-30, -1.0, math.nan):
        token, _ = run(z, u, least=least)
        for t in range(8):
            want = S.sample_row(z[t], float(u[t]), least=0.0 if math.isnan(least) else least)[0]
            assert int(token[t]) == want, (least, t)


@pytest.mark.parametrize("V", [100, 2500, 9000, 40000])
def test_ties(V):
    g = torch.Generator().manual_seed(V)
    u = torch.rand(12, generator=g)
    compare(torch.zeros(12, V), u, k=V // 3)  # one logit, cut by number
    compare(torch.zeros(12, V), u, p=0.37)
    compare(torch.zeros(12, V), u)
    few = torch.randint(0, 4, (12, V), generator=g).to(BF16)  # four logits
    for k in (1, V // 10, V // 2, V - 1):
        compare(few, u, k=k)
    for p in (0.1, 0.6, 0.9):
        compare(few, u, p=p)
    compare(few, u, k=V // 2, p=0.7, tau=3.0)


def test_many_logits_in_one_bin():
    g = torch.Generator().manual_seed(6)
    z = 5.0 + 1e-3 * torch.rand(6, 60000, generator=g)  # all in the first bin, thousands after splitting
    u = torch.rand(6, generator=g)
    compare(z, u, k=20000)
    compare(z, u, p=0.6)
    compare(z, u, k=41234, p=0.3)
    z[:, ::2] = 5.0
    compare(z, u, k=35000)


def test_tail_cuts():
    """k reaches tokens whose weights are 0."""
    z, u = make(4, 8000, F32, seed=7)
    z[:, 100:] -= 200.0
    for k in (90, 100, 101, 3000, 7999):
        compare(z, u, k=k)


def test_masked_tokens_and_rows():
    z, u = make(8, 5000, F32, seed=8)
    g = torch.Generator().manual_seed(9)
    gone = torch.rand(8, 5000, generator=g) < 0.7
    z[gone] = -math.inf
    z[1][gone[1]] = torch.finfo(F32).min
    z[2] = -math.inf
    z[3] = -math.inf
    z[3, 4321] = -5.0
    z[4, 7] = math.nan
    z[5, 11], z[5, 4000], z[5, 2222] = math.inf, math.inf, math.inf
    z[6] = torch.finfo(F32).min
    z[7, :] = torch.finfo(F32).max
    for kw in ({}, dict(k=40), dict(p=0.9), dict(k=1000, p=0.99, least=0.01), dict(tau=0.0)):
        token = compare(z, u, **kw)
        assert token[2] == -1 and token[4] == -1 and token[3] == 4321
        assert token[5] in (11, 2222, 4000)
        assert not any(bool(z[t, token[t]] == -math.inf) for t in (0, 1, 3, 5))


def test_without_logprobs_and_views_off_the_boundary():
    z, u = make(5, 3001, BF16, seed=10)
    want, _ = run(z, u, k=100)
    base = torch.empty(5 * 3001 + 3, dtype=BF16, device="cuda")
    base[3:] = z.view(-1).cuda()
    token = torch.empty(5, dtype=torch.int32, device="cuda")
    k = torch.full((5,), 100, dtype=torch.int32, device="cuda")
    B.moe_sample(base[3:].view(5, 3001), u.cuda(), token, top_k=k)
    assert torch.equal(token.cpu(), want)


def test_frequencies():
    V, n = 37, 20000
    z = torch.randn(1, V, generator=torch.Generator().manual_seed(11))
    u = (torch.arange(n) + 0.5) / n  # evenly spread numbers: each token gets its share, to one of them
    token, logprob = run(z.expand(n, V).contiguous(), u, tau=0.7)
    share = torch.softmax(z[0].double() / 0.7, 0)
    assert ((torch.bincount(token.long(), minlength=V) / n - share).abs() <= 1.0 / n + 1e-6).all()
    assert torch.allclose(logprob.double(), share.log()[token.long()], atol=1e-6)


def test_no_rows_and_refusals():
    e = torch.empty(0, device="cuda")
    B.moe_sample(torch.empty(0, 10, device="cuda"), e, e.int())
    z, u = torch.zeros(4, 20, device="cuda"), torch.zeros(4, device="cuda")
    token = torch.empty(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_sample(z[:, :10], u, token)
    with pytest.raises(TypeError, match="top_k"):
        B.moe_sample(z, u, token, top_k=u)
    with pytest.raises(ValueError, match="temperature"):
        B.moe_sample(z, u, token, temperature=u[:3])
    with pytest.raises(TypeError, match="logits"):
        B.moe_sample(z.double(), u, token)


def test_streams_and_repeats():
    z, u = make(30, 40000, BF16, seed=12)
    kw = dict(k=500, p=0.97)
    first = run(z, u, **kw)
    s = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s):
            again = run(z, u, **kw, stream=s)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_graph_replay_with_new_inputs():
    z, u = (t.cuda() for t in make(6, 9000, F32, seed=13))
    token, logprob = torch.empty(6, dtype=torch.int32, device="cuda"), torch.empty(6, device="cuda")
    p = torch.full((6,), 0.9, device="cuda")
    B.moe_sample(z, u, token, logprob, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_sample(z, u, token, logprob, top_p=p, stream=s)
    for seed in (14, 15):
        z2, u2 = make(6, 9000, F32, seed=seed)
        z.copy_(z2), u.copy_(u2)
        graph.replay()
        torch.cuda.synchronize()
        want = run(z2, u2, p=0.9)
        assert torch.equal(token.cpu(), want[0]) and torch.equal(logprob.cpu(), want[1])


def test_rows_past_32_bits():
    T, V = 16400, 131072  # over 2^31 logits
    z = torch.zeros(T, V, dtype=BF16, device="cuda")
    z[-1, 77777] = 60.0
    u = torch.full((T,), 0.5, device="cuda")
    token = torch.empty(T, dtype=torch.int32, device="cuda")
    B.moe_sample(z, u, token)
    assert int(token[-1]) == 77777 and bool((token[:-1] == 65536).all())
