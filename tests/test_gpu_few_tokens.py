"""The layer for 1 to 32 tokens on the GPU against its 64-bit values, within what its roundings allow: every
number of column tiles, heights of the down kernel's tiles, pieces of K that do not fill a stage, more experts than
a block counts at once, shared and repeated experts, pairs that are passed over."""

import pytest
import torch

import serve_ops_ref as S
import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(T, D, F, E, K, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

    x, w13, w2 = randn(T, D), randn(E, 2, F, D, std=D ** -0.5), randn(E, D, F, std=F ** -0.5)
    logits = torch.randn(T, E, generator=g, device="cuda")
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    return x, ids[:, :K].int().contiguous(), torch.softmax(top[:, :K], 1).contiguous(), w13, w2, logits


def workspace(x, w13, K):
    (T, D), (E, _, F, _) = x.shape, w13.shape
    ws = B.alloc_workspace(B.moe_few_workspace_bytes(T, D, F, E, K))
    return ws.fill_(0xA5)


def run(x, ids, scores, w13, w2, ws=None, stream=None):
    ws = workspace(x, w13, ids.shape[1]) if ws is None else ws
    out = torch.full_like(x, 7.0)
    B.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, out, ws, stream=stream)
    return out, B.moe_get_status(ws, stream) if stream is None else None


def compare(x, ids, scores, w13, w2, status=0):
    out, bits = run(x, ids, scores, w13, w2)
    assert bits == status
    R.check(out, *S.few(x, ids, scores, w13, w2), "out")
    return out


SIZES = [
    (1, 64, 64, 1, 1), (1, 128, 64, 4, 2), (1, 2048, 1408, 16, 6), (1, 7168, 2048, 10, 8), (2, 2496, 128, 8, 2),
    (3, 128, 64, 4096, 7), (5, 576, 320, 300, 5), (7, 192, 640, 257, 3), (8, 512, 512, 8, 8), (9, 1088, 192, 40, 3),
    (13, 256, 1088, 24, 4), (16, 4096, 256, 32, 8), (17, 320, 576, 20, 2), (24, 64, 2048, 64, 6),
    (32, 512, 256, 16, 16), (32, 1024, 448, 128, 8), (1, 64, 64, 600, 512), (4, 64, 128, 128, 128), (31, 640, 64, 3, 1),
]


@pytest.mark.parametrize("T,D,F,E,K", SIZES)
def test_against_64_bits(T, D, F, E, K):
    compare(*make(T, D, F, E, K, seed=T + D)[:5])


@pytest.mark.parametrize("T,K", [(1, 3), (8, 2), (16, 4), (32, 2)])
def test_all_pairs_on_one_expert(T, K):
    x, ids, scores, w13, w2, _ = make(T, 256, 128, 4, K, seed=1)
    compare(x, torch.full_like(ids, 3), scores, w13, w2)


def test_scores_in_bf16_and_of_either_sign():
    x, ids, scores, w13, w2, _ = make(6, 256, 192, 9, 3, seed=2)
    scores = (scores - 0.4).to(BF16)
    compare(x, ids, scores, w13, w2)


def test_repeated_experts_of_a_token_add_up():
    x, ids, scores, w13, w2, _ = make(10, 128, 64, 5, 4, seed=3)
    ids[:, 2] = ids[:, 0]
    ids[4] = ids[4, 0]
    compare(x, ids, scores, w13, w2)


def test_ids_outside_the_experts():
    x, ids, scores, w13, w2, _ = make(9, 128, 64, 5, 3, seed=4)
    for i, bad in enumerate((-1, 5, 2 ** 31 - 1, -2 ** 31)):
        ids[i, i % 3] = bad
    ids[7] = -1  # a token with none left
    out = compare(x, ids, scores, w13, w2, status=B.MOE_DEV_BAD_EXPERT_ID)
    assert not out[7].any()


def test_nothing_to_do():
    x, ids, scores, w13, w2, _ = make(4, 192, 64, 5, 2, seed=5)
    out, bits = run(x, torch.full_like(ids, -7), scores, w13, w2)
    assert bits == B.MOE_DEV_BAD_EXPERT_ID and not out.any()
    out, bits = run(x, ids, torch.zeros_like(scores), w13, w2)
    assert bits == 0 and not out.any()
    empty = torch.empty(0, 192, dtype=BF16, device="cuda")
    B.moe_routed_experts_fwd_few(empty, ids[:0], scores[:0], w13, w2, empty, B.alloc_workspace(256))


def test_pairs_with_a_score_of_zero_are_passed_over():
    x, ids, scores, w13, w2, _ = make(6, 128, 64, 6, 3, seed=6)
    ids = (ids % 5).contiguous()  # expert 5 belongs to the padding
    scores[2, 1] = -0.0
    ids[2, 1], scores[4], ids[4] = 5, 0.0, 5
    w13[5], w2[5] = float("nan"), float("inf")
    out = compare(x, ids, scores, w13, w2)
    assert not out[4].any()


def test_what_is_not_finite_stays_with_its_tokens():
    x, ids, scores, w13, w2, _ = make(12, 128, 64, 6, 2, seed=7)
    ids = torch.stack([torch.arange(12) % 3, 3 + torch.arange(12) % 2], 1).int().cuda()
    clean, _ = run(x, ids, scores, w13, w2)
    w13[2, 0, 5, 7], w2[4, 9, 3] = float("nan"), float("inf")
    x[0, 3] = float("nan")
    out, _ = run(x, ids, scores, w13, w2)
    hit = (ids[:, 0] == 2) | (torch.arange(12, device="cuda") == 0)
    assert torch.isnan(out[hit]).all()
    safe = ~hit
    cols = torch.arange(128, device="cuda") != 9
    assert torch.equal(out[safe][:, cols], clean[safe][:, cols])
    assert not torch.isfinite(out[safe & (ids[:, 1] == 4)][:, 9]).any()
    assert torch.equal(out[safe & (ids[:, 1] == 3)][:, 9], clean[safe & (ids[:, 1] == 3)][:, 9])


def test_near_the_large_forward():
    x, ids, scores, w13, w2, _ = make(32, 512, 256, 16, 4, seed=8)
    big = torch.empty_like(x)
    B.moe_routed_experts_fwd(x, ids, scores, w13, w2, big, B.alloc_workspace(B.moe_workspace_bytes(32, 512, 256, 16, 4)))
    out, _ = run(x, ids, scores, w13, w2)
    ref, bound = S.few(x, ids, scores, w13, w2)
    R.check(out, ref, bound, "few")
    # the large forward also rounds each pair's output: half a step of each
    assert float((out.float() - big.float()).norm() / big.float().norm()) < 2 * 2.0 ** -8 * 2


def choice(x, logits, w13, w2, K, normalize, stream=None):
    T = x.shape[0]
    ids, scores = torch.full((T, K), -9, dtype=torch.int32, device="cuda"), torch.full((T, K), -9.0, device="cuda")
    out, ws = torch.full_like(x, 7.0), workspace(x, w13, K)
    B.moe_layer_fwd_few(x, logits, w13, w2, ids, scores, out, ws, normalize=normalize, stream=stream)
    return ids, scores, out, B.moe_get_status(ws)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D,F,E,K", [(1, 256, 64, 64, 6), (1, 128, 64, 1, 1), (4, 64, 64, 256, 8), (11, 64, 128, 300, 40),
                                       (32, 128, 64, 7, 7), (3, 64, 64, 4096, 9)])
def test_from_logits(T, D, F, E, K, dtype, normalize):
    x, _, _, w13, w2, logits = make(T, D, F, E, K, seed=9)
    logits = logits.to(dtype)
    ids, scores, out, bits = choice(x, logits, w13, w2, K, normalize)
    wid, wsc = R.router_fwd(logits, K, normalize)
    assert torch.equal(ids.long(), wid) and bits == 0
    assert ((scores.double() - wsc).abs() <= wsc * R.router_rel(logits)).all()
    R.check(out, *S.few(x, ids, scores, w13, w2), "out")


def test_logits_that_tie_are_masked_or_not_numbers():
    x, _, _, w13, w2, logits = make(8, 64, 64, 40, 5, seed=10)
    logits = torch.round(logits)  # many ties
    logits[1] = 0.0
    logits[2, 3:] = -torch.inf
    logits[3] = -torch.inf
    logits[4, 7] = torch.nan
    logits[5, 0], logits[5, 9] = -0.0, 0.0
    logits[6] = torch.finfo(F32).min
    ids, scores, out, _ = choice(x, logits, w13, w2, 5, True)
    wid, wsc = torch.empty_like(ids), torch.empty_like(scores)
    B.moe_router_topk_fwd(logits, wid, wsc)
    assert torch.equal(ids, wid)
    assert torch.allclose(scores, wsc, rtol=1e-6, atol=0, equal_nan=True)
    assert not out[3].any() and torch.isnan(out[4]).all()
    good = torch.tensor([0, 1, 2, 3, 5, 6, 7], device="cuda")
    R.check(out[good], *S.few(x[good], ids[good], scores[good], w13, w2), "out")


def test_ids_written_by_the_kernel_before():
    """The down kernel reads ids before it waits for the gate/up kernel: they have to be the call's own."""
    x, _, _, w13, w2, _ = make(4, 512, 256, 32, 4, seed=11)
    g = torch.Generator(device="cuda").manual_seed(12)
    all_logits = torch.randn(40, 4, 32, generator=g, device="cuda")
    ids, scores = torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.zeros(4, 4, device="cuda")
    ws, outs = workspace(x, w13, 4), []
    for z in all_logits:
        out = torch.empty_like(x)
        B.moe_router_topk_fwd(z, ids, scores)
        B.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, out, ws)
        outs.append(out)
    for z, out in zip(all_logits, outs):
        B.moe_router_topk_fwd(z, ids, scores)
        torch.cuda.synchronize()
        again, _ = run(x, ids, scores, w13, w2)
        assert torch.equal(out, again)


def test_two_streams_at_once():
    a, b = make(8, 1024, 256, 32, 4, seed=13)[:5], make(3, 512, 512, 16, 6, seed=14)[:5]
    want = [run(*a)[0], run(*b)[0]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    spaces = [workspace(a[0], a[3], 4), workspace(b[0], b[3], 6)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (args, s) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(s):
                outs[i].append(run(*args, ws=spaces[i], stream=s)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_graph_replay_with_new_inputs():
    x, ids, scores, w13, w2, logits = make(5, 256, 128, 24, 3, seed=15)
    ws, out, out2 = workspace(x, w13, 3), torch.empty_like(x), torch.empty_like(x)
    ids2, scores2 = torch.empty_like(ids), torch.empty_like(scores)
    run(x, ids, scores, w13, w2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_routed_experts_fwd_few(x, ids, scores, w13, w2, out, ws, stream=s)
        B.moe_layer_fwd_few(x, logits, w13, w2, ids2, scores2, out2, ws, stream=s)
    for seed in (16, 17):
        x2, i2, s2, _, _, l2 = make(5, 256, 128, 24, 3, seed=seed)
        x.copy_(x2), ids.copy_(i2), scores.copy_(s2), logits.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run(x2, i2, s2, w13, w2)[0])
        assert torch.equal(ids2, i2) and torch.equal(out2, choice(x2, l2, w13, w2, 3, True)[2])


def test_repeats_give_the_same_bits():
    args = make(32, 1024, 448, 128, 8, seed=18)[:5]
    first, _ = run(*args)
    for _ in range(5):
        assert torch.equal(run(*args)[0], first)


def test_weights_past_32_bits():
    T, D, F, E, K = 2, 1024, 1024, 1100, 2  # over 2^31 elements of w13
    w13 = torch.zeros(E, 2, F, D, dtype=BF16, device="cuda")
    w2 = torch.zeros(E, D, F, dtype=BF16, device="cuda")
    x, _, scores, s13, s2, _ = make(T, D, F, 2, K, seed=19)
    at = torch.tensor([[3, 1099], [1099, 1023]], dtype=torch.int32, device="cuda")
    for e, src in ((3, 0), (1099, 1), (1023, 0)):
        w13[e], w2[e] = s13[src], s2[src]
    out, _ = run(x, at, scores, w13, w2)
    same = torch.tensor([[0, 1], [1, 0]], dtype=torch.int32, device="cuda")
    R.check(out, *S.few(x, same, scores, s13, s2), "out")


@pytest.mark.parametrize("T,K", [(15, 8), (31, 16)])
def test_experts_with_every_number_of_tokens(T, K):
    x, _, scores, w13, w2, _ = make(T, 192, 128, T, K, seed=11)
    chosen = [[] for _ in range(T)]
    for count in range(T, 0, -1):  # expert count - 1 goes to the tokens with the fewest so far: T (T + 1) / 2 pairs
        for t in sorted(range(T), key=lambda t: (len(chosen[t]), t))[:count]:
            chosen[t].append(count - 1)
    ids = torch.tensor(chosen, dtype=torch.int32, device="cuda")
    assert ids.shape == (T, K)
    compare(x, ids, scores, w13, w2)
