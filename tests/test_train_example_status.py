"""The training example without a GPU: an error of any step's calls ends the training."""

import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_moe_lm.py")


@pytest.fixture
def ex():
    spec = importlib.util.spec_from_file_location("train_moe_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Model:
    """Reports the given status words, one per step, each cleared by the next step's calls."""
    T, V = 4, 8

    def __init__(self, words):
        self.words, self.params, self.steps = words, {}, 0

    def forward_backward(self, tokens, targets=None, teacher=None, temperature=1.0):
        self.steps += 1
        return torch.ones(self.T)

    def status(self):
        return self.words[self.steps - 1]


@pytest.mark.parametrize("words", [[0, 2, 0, 0], [2, 0, 0, 0], [0, 0, 0, 4]])
def test_an_error_of_any_step_ends_the_training(ex, monkeypatch, words):
    model = Model(words)
    monkeypatch.setattr(ex, "MoeLm", lambda **kw: model)
    monkeypatch.setattr(ex, "batch", lambda T, V, seed: (torch.zeros(T), torch.zeros(T)))
    with pytest.raises(RuntimeError, match="status"):
        ex.train(len(words))
    assert model.steps == 1 + next(i for i, w in enumerate(words) if w)
