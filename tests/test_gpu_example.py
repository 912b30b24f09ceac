"""The example that trains a small mixture-of-experts model with this library's
operators and then serves it (needs an MI355X)."""
import importlib.util
import math
import os

import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_and_serve", os.path.join(ROOT, "examples", "train_and_serve.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_learns_and_answers(example):
    losses, right = example.main(["--steps", "60", "--tokens", "2048"])
    assert abs(losses[0] - math.log(example.VOCAB)) < 0.5
    assert losses[-1] < 0.5 and right >= 0.95


def test_gradients_of_the_experts(example):
    """The step's expert gradients (through vocab_cross_entropy, fwd and wgrad,
    MXFP8 operands) point along those of the same layer in float64."""
    model = example.Model(seed=3)
    words = torch.randint(0, example.VOCAB, (512,), device="cuda")
    targets = example.next_word(words)
    seen = []
    ortho, mxw.orthogonalize = mxw.orthogonalize, lambda m: seen.append(m.clone()) or torch.zeros_like(m)
    try:
        gate_up, down = (t.double().requires_grad_() for t in (model.gate_up, model.down))
        vocabulary = model.words.to(torch.bfloat16).double()
        loss = model.step(words, targets, 0.0)
    finally:
        mxw.orthogonalize = ortho
    x = model.embedding[words]
    ids, w = model.routing(x)
    x = x.double()
    y = x.clone()
    for e in range(example.EXPERTS):
        gu = x @ gate_up[e].t()
        h = torch.nn.functional.silu(gu[:, :example.WIDTH]) * gu[:, example.WIDTH:]
        y = y + (w.double() * (ids == e)).sum(1, keepdim=True) * (h @ down[e].t())
    ref = torch.nn.functional.cross_entropy(y @ vocabulary.t(), targets)
    ref.backward()
    assert abs(loss.item() - ref.item()) < 0.02
    for got, want in zip(seen, (gate_up.grad, down.grad)):
        cos = (got.double() * want).sum() / (got.double().norm() * want.norm())
        assert cos > 0.99
