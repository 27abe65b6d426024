"""The FP64 oracle of the training-step operators, pinned by finite differences and by facts
that the formulas fix on their own."""

import numpy as np
import pytest

from oracle import training_oracle as T


def _rng(seed):
    return np.random.default_rng(seed)


def _diff(f, a, direction, h=1e-5):
    """Central difference of f along a direction."""
    return (f(a + h * direction) - f(a - h * direction)) / (2 * h)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 7])
def test_norm_gradients_are_the_forwards_slopes(post, gate_rows):
    """For L = <h, dh> + <x', dx'> each gradient's product with a direction is the slope of L
    along it (central differences, step 1e-5: error about 1e-10 of the second derivatives)."""
    rng = _rng(1 + gate_rows)
    M, d, s, eps = 7, 6, 0.7, 1e-3
    x, y, dh, dxo = (rng.standard_normal((M, d)) for _ in range(4))
    w_post, w_pre = rng.standard_normal(d) + 1, rng.standard_normal(d) + 1
    gate = rng.standard_normal((-(-M // gate_rows), d)) if gate_rows else None

    def L(x=x, y=y, w_post=w_post, gate=gate, w_pre=w_pre):
        xo, h = T.norm_residual_fwd(x, y, post, w_post if post else None, gate, gate_rows, w_pre, s, eps)
        return np.sum(h * dh) + np.sum(xo * dxo)

    xo, _ = T.norm_residual_fwd(x, y, post, w_post if post else None, gate, gate_rows, w_pre, s, eps)
    g, mag = T.norm_residual_bwd(xo, y, dh, dxo, post, w_post if post else None, gate, gate_rows, w_pre, s, eps)
    named = dict(x=x, y=y, w_pre=w_pre)
    if post:
        named["w_post"] = w_post
    if gate is not None:
        named["gate"] = gate
    assert set(g) == {"d" + k for k in named}
    for k, v in named.items():
        for _ in range(3):
            v_dir = rng.standard_normal(v.shape)
            slope = _diff(lambda a: L(**{k: a}), v, v_dir)  # noqa: B023
            assert abs(np.sum(g["d" + k] * v_dir) - slope) <= 1e-6 * (1 + abs(slope)), k
        assert np.all(np.abs(g["d" + k]) <= mag["d" + k] * (1 + 1e-12)), k


@pytest.mark.parametrize("smoothing", [0.0, 0.2])
def test_preference_gradient_is_the_loss_slope(smoothing):
    rng = _rng(5)
    P, S, V = 2, 4, 5
    x = rng.standard_normal((2 * P, S, V))
    labels = rng.integers(0, V, (2 * P, S))
    labels[0, :2] = -100
    labels[3, 1] = V
    ref = rng.standard_normal((2 * P, S))
    loss, D, lp, d, _ = T.preference_loss(x, labels, ref, 0.5, smoothing, grad_scale=3.0)
    for _ in range(4):
        v = rng.standard_normal(x.shape)
        slope = _diff(lambda a: 3.0 * T.preference_loss(a, labels, ref, 0.5, smoothing)[0], x, v)  # noqa: B023
        assert abs(np.sum(d * v) - slope) <= 1e-7
    assert np.all(d[0, :2] == 0) and np.all(d[3, 1] == 0)
    assert np.allclose(d.sum(axis=2), 0, atol=1e-12)  # softmax gradients have no mean


def test_preference_facts():
    """No difference to the reference gives log 2; an empty answer counts as 0."""
    x = _rng(6).standard_normal((2, 3, 4))
    labels = np.array([[0, 1, 2], [3, 2, 1]])
    ref = T.token_logps(x, labels)
    assert abs(T.preference_loss(x, labels, ref, 0.1)[0] - np.log(2)) <= 1e-12
    assert np.allclose(np.exp(T.token_logps(np.repeat(x[:1, :1], 4, 1), np.array([[0, 1, 2, 3]]))).sum(), 1)
    labels[1] = -100
    assert T.preference_loss(x, labels, None, 0.1)[1][1] == 0


def test_clip_facts():
    g = [np.array([3.0]), np.array([[4.0]]), np.zeros(0)]
    assert T.grad_norm(g) == 5.0
    assert T.clip_coefficient(5.0, 10.0) == 1.0
    assert abs(T.clip_coefficient(5.0, 1.0) - 0.2) <= 1e-7
