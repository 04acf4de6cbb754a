"""The example that trains a small model with every operator: its gradients against torch's in 64 bits,
and its loss going down."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_moe_lm.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("train_moe_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(model, tokens, targets, teacher, temperature):
    """The same model and loss in 64 bits with the choices of experts that the step made; its gradients."""
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in model.params.items()}
    ids = model.ids.cpu().long()
    norm = lambda h, i: torch.nn.functional.layer_norm(h, (model.D,), p[f"gamma{i}"], p[f"beta{i}"])
    h0 = p["embedding"][tokens.cpu()]
    n1 = norm(h0, 1)
    scores = torch.softmax((n1 @ p["router"].T).gather(1, ids), 1)
    out = 0.0
    for k in range(model.K):
        gate, up = torch.einsum("tfd,td->tf", p["w13"][ids[:, k], 0], n1), torch.einsum(
            "tfd,td->tf", p["w13"][ids[:, k], 1], n1)
        out = out + scores[:, k:k + 1] * torch.einsum("tdf,tf->td", p["w2"][ids[:, k]],
                                                      torch.nn.functional.silu(gate) * up)
    z = norm(h0 + out, 2) @ p["head"].T
    if teacher is None:
        loss = torch.nn.functional.cross_entropy(z, targets.cpu().long(), reduction="none")
    else:
        t = torch.softmax(teacher[1].cpu().double() / temperature, 1)
        q = torch.log_softmax(z / temperature, 1).gather(1, teacher[0].cpu().long())
        loss = temperature ** 2 * (t * (t.log() - q)).sum(1)
    grads = torch.autograd.grad(loss.mean(), list(p.values()))
    return loss.detach(), dict(zip(p, grads))


@pytest.mark.parametrize("distill", [False, True])
def test_step_gradients(ex, distill):
    model = ex.MoeLm(tokens=150, hidden=128, ffn=64, experts=4, top_k=2, vocab=300, seed=3)
    tokens, targets = ex.batch(150, 300, seed=5)
    targets[::11] = -100
    teacher = ex.teacher_of(targets.clamp(min=0), 300, 5, seed=6) if distill else None
    loss = model.forward_backward(tokens, targets, teacher, 2.0)
    assert model.status() == 0
    want, grads = reference(model, tokens, targets, teacher, 2.0)
    # a gradient passes some ten bf16 roundings (each output and intermediate of the seven operators), each
    # off by at most 2^-8 of its value; the losses see the roundings of n1, the experts, h1 and n2
    for name, g in grads.items():
        got = model.grads[name].double().cpu()
        assert float((got - g).norm() / g.norm()) < 10 * 2.0 ** -8, name
    assert float((loss.double().cpu() - want).norm() / want.norm()) < 6 * 2.0 ** -8


@pytest.mark.parametrize("distill", [False, True])
def test_loss_goes_down(ex, distill):
    losses = ex.train(60, distill, tokens=512, hidden=128, ffn=128, experts=4, vocab=256)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert last < 0.7 * first, (first, last)
