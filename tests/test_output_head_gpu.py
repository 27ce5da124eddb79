"""The output head's operators together, as examples/output_head.py runs them."""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(tg):
    spec = importlib.util.spec_from_file_location("output_head", os.path.join(ROOT, "examples", "output_head.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_one_step_against_autograd_in_64_bits(example):
    """Gradients of the whole chain: each passes at most five roundings to
    bf16 (y, G, dy, xh's inputs are exact, the result) of relative size 2^-9 on
    average, errors of either sign: 2 % of the norm is four times their sum."""
    v, d, t = 1500, 264, 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    directions = torch.randn(v, d, device="cuda", generator=gen)
    x, target = example.batch(directions, t, gen)
    head = example.OutputHead(v, d)
    head.weight.add_(torch.randn(d, device="cuda", generator=gen).to(x.dtype) * 0.2)
    loss, dx = head.loss_and_gradients(x, target)
    xs, w, b, p = (q.detach().double().requires_grad_() for q in (x, head.weight, head.bias, head.proj))
    y = torch.nn.functional.layer_norm(xs, (d,), w, b, head.EPS)
    want = torch.nn.functional.cross_entropy(y @ p.T, target, ignore_index=-100)
    want.backward()
    assert abs(float(loss) - float(want)) < 2e-3 * float(want)
    for got, ref in ((dx, xs), (head.grads[0], w), (head.grads[1], b), (head.grads[2], p)):
        assert rel(got, ref.grad) < 0.02


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_training_learns(example, dtype, bits):
    v, d, t = 512, 256, 1024
    gen = torch.Generator(device="cuda").manual_seed(5)
    directions = torch.randn(v, d, device="cuda", generator=gen)
    head = example.OutputHead(v, d, dtype, bits)
    losses = []
    for _ in range(25):
        x, target = example.batch(directions, t, gen)
        loss, _ = head.loss_and_gradients(x.to(dtype), target)
        head.update(lr=2e-2)
        losses.append(float(loss))
    # an untrained head is near log(v) (its logits have a deviation of 0.3),
    # a trained one tells 512 well separated directions apart
    assert abs(losses[0] - math.log(v)) < 0.3
    assert losses[-1] < 0.1 * losses[0]
    assert all(math.isfinite(x) for x in losses)
