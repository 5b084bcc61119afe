"""The example that trains a layer norm and a vocabulary projection: its
gradients against the same model in 64 bits, the loss falling with 8-bit and
32-bit moments alike, and an overflowed step skipped."""
import importlib.util
import math
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("train_head", os.path.join(ROOT, "examples", "train_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_of_the_whole_path():
    """dx, d ln_weight, d ln_bias, d weight against autograd in 64 bits.  The
    path rounds y, G, dy and each result to bfloat16 (2^-8 each, independent
    errors): 2^-6 of a gradient's norm covers the four."""
    M = _example()
    h = M.Head(vocab=700, hidden=136, tokens=90, bits=32, loss_scale=64.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    for k in ("ln_weight", "ln_bias"):
        h.master[k] += 0.1 * torch.randn(136, device="cuda", generator=g)
        h.param[k].copy_(h.master[k])
    x, t = next(M.batches(700, 136, 90))
    loss, total = h.forward(x, t)
    dx = h.backward(x, t)
    p = {k: v.double().requires_grad_() for k, v in h.param.items()}
    x64 = x.double().requires_grad_()
    y = torch.nn.functional.layer_norm(x64, (136,), p["ln_weight"], p["ln_bias"], 1e-5)
    want = torch.nn.functional.cross_entropy(y @ p["weight"].t(), t, ignore_index=-100)
    # the loss: y's rounding moves a logit by 2^-9 sum |y w| / sqrt(terms) at most a few times over
    assert abs(float(total[0]) - float(want.detach())) < 0.01 * float(want.detach())
    (64.0 * want).backward()
    for got, ref in ((dx, x64.grad), (h.grad["ln_weight"], p["ln_weight"].grad), (h.grad["ln_bias"], p["ln_bias"].grad),
                     (h.grad["weight"], p["weight"].grad)):
        assert (got.double() - ref).norm() <= 2.0 ** -6 * ref.norm()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_loss_falls(bits, dtype):
    M = _example()
    losses = M.main(["--steps", "40", "--vocab", "2000", "--hidden", "256", "--tokens", "1024", "--bits", str(bits),
                     "--dtype", dtype])
    assert abs(losses[0] - math.log(2000)) < 0.5
    assert losses[-1] < 0.5 * losses[0]


def test_8_and_32_bit_moments_train_alike():
    M = _example()
    a, b = (M.main(["--steps", "60", "--vocab", "1500", "--hidden", "192", "--tokens", "1024", "--bits", n]) for n in ("8", "32"))
    assert abs(a[-1] - b[-1]) < 0.15 * b[0]


def test_overflowed_step_is_skipped():
    M = _example()
    h = M.Head(vocab=300, hidden=64, tokens=50, dtype="fp16", bits=8, loss_scale=2.0 ** 40)
    before = {k: w.clone() for k, w in h.master.items()}
    x, t = next(M.batches(300, 64, 50, "fp16"))
    h.forward(x, t)
    h.backward(x, t)
    assert not h.update() and h.scale == 2.0 ** 39 and h.t == 0
    for k, w in h.master.items():
        assert torch.equal(w, before[k])


def test_8_and_32_bit_moments_end_at_the_same_loss():
    """8-bit moments are off by a thirtieth of themselves at random, so the
    steps are, and the training ends at 32-bit moments' loss: within a quarter of it."""
    M = _example()
    a, b = (M.main(["--steps", "120", "--vocab", "1500", "--hidden", "192", "--tokens", "1024", "--bits", n]) for n in ("8", "32"))
    a, b = (sum(x[-10:]) / 10 for x in (a, b))
    assert abs(a - b) <= 0.25 * b + 0.02
