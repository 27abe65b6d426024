"""The example that runs the training-step operators together: its loss starts at log 2 (the
adapters begin as the identity, so the model is its own reference) and falls, and one of its
gradients is checked against a difference of the loss through the whole model."""

import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_preference_example_learns(gpu_lib):
    import preference_step as E

    losses, norms = E.train(steps=12, report=lambda s: print(s, flush=True))
    # both passes run the same kernels on the same adapters' products (B = 0): equal bits, D = 0
    assert losses[0] == pytest.approx(math.log(2), abs=1e-6)
    assert losses[-1] < 0.5 * losses[0]
    assert all(math.isfinite(n) and n > 0 for n in norms)


def test_example_gradient_is_the_slope(gpu_lib):
    """d loss along the gradient of the head's B: its kernels see BF16 activations, so the change of
    the loss over a step of the direction g / |g| is compared within 5% of |g|, the sum of the
    chain's BF16 roundings (seven of 2^-8)."""
    import bit_nf4_quantized_dq_amd as Q
    import preference_step as E

    model = E.Model()
    tokens, labels = E.batch(model)
    ref = Q.token_logps(model.forward(tokens, adapted=False)[0], labels)
    logits, saved = model.forward(tokens)
    _, _, _, d = Q.preference_loss(logits, labels, ref, 0.1)
    g = model.backward(d, saved)[7].float()
    B0, e = model.B[3].clone(), 0.05

    def loss(sign):
        model.B[3].copy_((B0.float() + sign * e * g / g.norm()).to(torch.bfloat16))
        return float(Q.preference_loss(model.forward(tokens)[0], labels, ref, 0.1, need_grad=False)[0])

    slope = (loss(1) - loss(-1)) / (2 * e)
    assert abs(slope - float(g.norm())) <= 0.05 * float(g.norm())
