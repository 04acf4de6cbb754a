"""The top-k router on the GPU: ids exactly those of a stable sort, scores and gradients against their
64-bit values, masked and broken rows, and the way through the expert layer's own gradient."""

import pytest
import torch

import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rand(*shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def fwd(z, K, normalize, stream=None):
    T = z.shape[0]
    ids = torch.full((T, K), -7, dtype=torch.int32, device="cuda")
    scores = torch.full((T, K), 7.0, device="cuda")
    B.moe_router_topk_fwd(z.cuda(), ids, scores, normalize, stream=stream)
    return ids, scores


def bwd(z, ids, ds, normalize):
    dz = torch.full(z.shape, 7.0, dtype=z.dtype, device="cuda")
    B.moe_router_topk_bwd(z.cuda(), ids.int().cuda(), ds.cuda(), dz, normalize)
    return dz


def compare(z, K, normalize, seed):
    ids, scores = fwd(z, K, normalize)
    want_ids, want = R.router_fwd(z, K, normalize)
    assert torch.equal(ids.cpu().long(), want_ids)
    rel = R.router_rel(z)
    R.check(scores, want, rel * want + 2.0 ** -126, "scores")
    ds = rand(z.shape[0], K, seed=seed)
    got = bwd(z, want_ids, ds, normalize)
    ref, mag = R.router_bwd(z, want_ids, ds, normalize)
    R.check(got, ref, 3 * rel * mag + R.round_bound(ref, z.dtype) + 2.0 ** -126, "dlogits")


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 2, 2), (3, 8, 2), (257, 64, 6), (129, 128, 8), (65, 130, 3), (100, 256, 8),
                                   (9, 257, 1), (33, 512, 40), (7, 1000, 10), (6, 1024, 1), (5, 1025, 4), (3, 4096, 33),
                                   (2, 4095, 8), (4, 48, 48)])
def test_choice_scores_and_gradient(T, E, K, dtype, normalize):
    compare(rand(T, E, seed=T * 7919 + E, dtype=dtype), K, normalize, seed=E + K)


@pytest.mark.parametrize("E", [5, 64, 200, 2000])
def test_equal_logits_go_to_the_lowest_expert(E):
    z = torch.zeros(6, E)
    z[1] = -0.0
    z[2, ::2] = -0.0  # minus zero equals zero
    z[3] = torch.arange(E).float() // 3
    z[4, -1] = 1.0
    for normalize in (True, False):
        compare(z, min(E, 5), normalize, seed=3)


def test_masked_experts():
    z = rand(5, 40, seed=4)
    z[0, 3:] = -torch.inf  # three left for eight places
    z[1, 1:] = -torch.inf
    z[2] = -torch.inf      # none left
    z[3, ::2] = torch.finfo(F32).min
    for normalize in (True, False):
        compare(z, 8, normalize, seed=5)
        ids, scores = fwd(z, 8, normalize)
        assert not scores[2].any() and torch.equal(ids[2].cpu(), torch.arange(8, dtype=torch.int32))
        assert not scores[0, 3:].any() and not scores[1, 1:].any()
        assert not bwd(z, ids, torch.ones(5, 8), normalize)[2].any()


def test_a_broken_row_shows_and_stays_alone():
    z = rand(4, 64, seed=6)
    want = fwd(z, 4, True)
    z[1, 10] = float("nan")
    for normalize in (True, False):
        ids, scores = fwd(z, 4, normalize)
        assert ids[1, 0] == 10 and torch.isnan(scores[1]).all() and not torch.isnan(scores[[0, 2, 3]]).any()
    ids, scores = fwd(z, 4, True)
    keep = [0, 2, 3]
    assert torch.equal(ids[keep], want[0][keep]) and torch.equal(scores[keep], want[1][keep])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_nan_of_either_sign_sorts_above_all(dtype):
    z = rand(3, 64, seed=16, dtype=dtype)
    z[0, 9] = torch.inf
    z[0, 20] = float("nan")
    z[1, 30] = -torch.tensor(float("nan"), dtype=dtype)
    z[1, 31] = torch.copysign(torch.tensor(float("nan"), dtype=dtype), torch.tensor(-1.0, dtype=dtype))
    for normalize in (True, False):
        ids, scores = fwd(z, 3, normalize)
        assert ids[0].tolist()[:2] == [20, 9] and ids[1].tolist()[:2] == [30, 31]
        assert torch.isnan(scores[:2]).all() and not torch.isnan(scores[2]).any()


@pytest.mark.parametrize("E,K", [(256, 8), (200, 40), (64, 1)])
def test_logits_that_differ_only_in_their_last_bits(E, K):
    # closer than the upper 24 bits tell, in and at the edge of the choice, in ascending and mixed order
    near = 1.0 + torch.arange(E, dtype=torch.float64) * 2.0 ** -23
    z = torch.stack([near, near.flip(0), near[torch.randperm(E, generator=torch.Generator().manual_seed(1))],
                     torch.cat([4 + torch.arange(K, dtype=torch.float64), near[K:]])]).float()
    for normalize in (True, False):
        compare(z, K, normalize, seed=17)


def test_ids_outside_are_passed_over():
    z, ds = rand(2, 16, seed=7), torch.ones(2, 3)
    ids = torch.tensor([[4, -1, 16], [2, 1 << 30, 5]], dtype=torch.int32)
    got = bwd(z, ids, ds, True)
    full = torch.zeros(2, 16)
    assert got[0, 4] == 0 and not got[0].any()  # one expert chosen: its score is 1 whatever its logit
    full[1, [2, 5]] = 1.0
    assert not got[1][full[1].cuda() == 0].any()


def test_large_rows_pass_32_bits():
    T, E = 2 ** 20 + 1, 2048 + 4
    z = torch.zeros(T, E, dtype=BF16, device="cuda")  # over 2^31 elements
    z[-1, 7] = 1.0
    ids = torch.empty(T, 2, dtype=torch.int32, device="cuda")
    scores = torch.empty(T, 2, device="cuda")
    B.moe_router_topk_fwd(z, ids, scores)
    assert ids[-1].tolist() == [7, 0] and ids[-2].tolist() == [0, 1]


def test_no_rows_and_refusals():
    ids, scores = fwd(torch.zeros(0, 8), 2, True)
    with pytest.raises(B.MoeError):
        fwd(torch.zeros(2, 8), 9, True)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_router_topk_fwd(torch.zeros(4, 16, device="cuda")[:, :8], ids, scores)


def test_gradient_is_the_difference_of_the_forward():
    z, v, ds = rand(8, 64, seed=8), rand(8, 64, seed=9), rand(8, 4, seed=10)
    ids, _ = fwd(z, 4, False)
    h = 1e-3  # small enough that the order of the first four stays
    up, down = (fwd(z + s * h * v, 4, False) for s in (1, -1))
    assert torch.equal(up[0], ids) and torch.equal(down[0], ids)
    diff = ((up[1].double() - down[1].double()) * ds.cuda().double()).sum() / (2 * h)
    got = (bwd(z, ids, ds, False).double() * v.cuda().double()).sum()
    assert abs(float(diff - got)) < 8 * 4 * (h * h * 100 + 2.0 ** -22 / h)
