"""The norms around a block with rows shorter than a 16-byte piece, anywhere in memory: values right, nothing of the
neighbours used or written (which pieces are read is tests/test_row_pieces.py's). And the pieces at the ends of longer
rows, in groups of every size."""

import pytest
import torch

import block_norm_ref as N
import train_ops_ref as R
from mixture_experts_routed_topk_gb300 import binding as B
from test_gpu_block_norm import EPS, NAMES, back, make, rand

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


class Amid:
    """Tensors on the GPU, each in the middle of a buffer of NaN, `offset` elements behind a 16-byte boundary."""

    def __init__(self, offset):
        self.offset, self.kept = offset, []

    def __call__(self, t, blank=False):
        if t is None:
            return None
        base = torch.full((t.numel() + 64 + self.offset,), float("nan"), dtype=t.dtype, device="cuda")
        assert base.data_ptr() % 16 == 0
        at = slice(32 + self.offset, 32 + self.offset + t.numel())
        if not blank:
            base[at] = t.reshape(-1).cuda()
        self.kept.append((base, at))
        return base[at].view(t.shape)

    def check_around(self):
        for base, at in self.kept:
            assert torch.isnan(base[:at.start]).all() and torch.isnan(base[at.stop:]).all()


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7, 9])
def test_short_rows(D, dtype, offset, gate):
    for T in (1, 2, 3, 5, 20, 40, 5000):
        c = make(T, D, dtype, dtype, gate=gate)
        args = [c[k] for k in ("block", "residual", "post_gamma", "gate", "pre_gamma")]
        amid = Amid(offset)
        dev = [amid(t) for t in args]
        got = [amid(c["block"], True), amid(c["block"], True), torch.full((T,), 7.0, device="cuda"),
               torch.full((T,), 7.0, device="cuda")]
        B.moe_block_norm_fwd(*dev, *got, residual_scale=0.7, eps=EPS)
        want, bounds = N.fwd(*args, 0.7, EPS, True), N.fwd_bounds(*args, 0.7, EPS, True, dtype)
        for name, g, w, b in zip(("stream", "normed", "post_rstd", "pre_rstd"), got, want, bounds):
            R.check(g, w, b, f"{name} T={T}")

        a = dict(dstream=rand(T, D, seed=60, dtype=dtype), dnormed=rand(T, D, seed=61, dtype=dtype), block=c["block"],
                 stream=want[0].to(dtype), post_gamma=c["post_gamma"], gate=c["gate"], pre_gamma=c["pre_gamma"],
                 post_rstd=want[2].float(), pre_rstd=want[3].float())
        grads = dict(dblock=c["block"], dresidual=c["block"], dpost_gamma=c["post_gamma"], dgate=c["gate"],
                     dpre_gamma=c["pre_gamma"])
        dev = [t.cuda() if k.endswith("rstd") else amid(t) for k, t in a.items()]
        out = [amid(grads[k], True) for k in NAMES]
        B.moe_block_norm_bwd(*dev, *out, B.alloc_workspace(B.moe_block_norm_bwd_workspace_bytes(T, D)),
                             residual_scale=0.7)
        ref, errs = N.bwd(*a.values(), 0.7)
        for name, g, w, e in zip(NAMES, out, ref, errs):
            R.check(g, w, e + R.round_bound(w, g.dtype), f"{name} T={T}")
        amid.check_around()


@pytest.mark.parametrize("dtype", [F32, BF16, F16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [13, 121, 505, 519, 777, 1017, 1501, 2041, 3001, 4089, 4103, 6001, 8185])
def test_first_and_last_chunks_of_every_group(D, dtype):
    """Column sums of groups of 32 to 512 threads, several to a block, whose rows all lie differently to 16-byte pieces."""
    for T in (15, 70):
        c = make(T, D, dtype, F32, gate="channel", seed=3)
        a, got = back(c, F32, True, 0.7)
        want, errs = N.bwd(*a.values(), 0.7)
        for name, w, e in zip(NAMES, want, errs):
            R.check(got[name], w, e + R.round_bound(w, got[name].dtype), f"{name} T={T}")
