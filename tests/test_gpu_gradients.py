"""GPU parity of the gradient norm, clipping and the clipped optimizer step against the oracle.

Tolerances: squares and sums are FP64 (errors below 1e-12 at these sizes), the norm is rounded
to FP32 once (u = 2^-24).  The coefficient max_norm / (norm + 1e-6) adds three roundings, the
product one, and BF16 results one of 2^-8.  The clipped step is adamw_step on FP32 gradients
that carry the coefficient's error (4u relative): beside the bounds of the plain step
(test_gpu_adamw) m and v move by 8u of their gradient terms and the step by its share."""

import numpy as np
import pytest
import torch

import oracle as O
from bit_nf4_quantized_dq_amd import inputs as I
from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
U, UB = 2.0**-24, 2.0**-8
BF, F32 = torch.bfloat16, torch.float32


def _tensors(sizes, types, seed=0, std=1e-3, shift=0):
    """Tensors back to back in one buffer of each type, `shift` elements from its start: any
    alignment of their elements."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n, t in zip(sizes, types):
        base = torch.empty(n + shift + 1, dtype=t, device="cuda")
        v = base[shift:shift + n]
        v.copy_((std * torch.randn(n, generator=g)).to(t))
        out.append(v)
    return out


def _np(ts):
    return [t.double().cpu().numpy() for t in ts]


SIZES = [1, 7, 8, 9, 511, 512, 4095, 4096, 4097, 16383, 16384, 16385, 0, 100003, 3]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("types", ["bf16", "f32", "mixed"])
def test_norm_and_clip(gpu_lib, shift, types):
    import bit_nf4_quantized_dq_amd as Q

    kinds = {"bf16": [BF] * 15, "f32": [F32] * 15, "mixed": [BF, F32] * 7 + [BF]}[types]
    g = _tensors(SIZES, kinds, seed=shift, shift=shift)
    ref = T.grad_norm(_np(g))
    for out_types in (None, [BF] * 15, [F32] * 15):
        out = None if out_types is None else _tensors(SIZES, out_types, shift=(shift + 1) % 4)
        work = [t.clone() for t in g] if out is None else g
        gl = Q.GradList(work, out=out)
        norm = Q.grad_norm(gl)
        max_norm = float(np.float32(0.3 * ref))
        before = Q.grad_clip(gl, max_norm)
        torch.cuda.synchronize()
        assert abs(float(norm) - ref) <= 2 * U * ref and torch.equal(norm, before)
        c = T.clip_coefficient(float(norm), max_norm)
        for a, b in zip(_np(g), out if out is not None else work):
            r = UB if b.dtype == BF else U
            assert np.all(np.abs(b.double().cpu().numpy() - c * a) <= (r + 4 * U) * np.abs(c * a) + 1e-40)
        # already below the limit: copied, or left alone, exactly
        before = Q.grad_clip(gl, 1e9)
        torch.cuda.synchronize()
        src = g if out is not None else work
        for a, b in zip(src, out if out is not None else work):
            assert torch.equal(a.to(b.dtype), b)


def test_one_element_and_one_large_tensor(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    for n in (1, 5, 1023, 9_000_001):
        print(f"grad norm n={n}", flush=True)
        g = _tensors([n], [BF], seed=n)
        norm = Q.grad_norm(Q.GradList(g))
        torch.cuda.synchronize()
        ref = T.grad_norm(_np(g))
        assert abs(float(norm) - ref) <= 2 * U * ref


def test_nothing_overflows_or_vanishes_on_the_way(gpu_lib):
    """Squares beyond FP32's range in both directions."""
    import bit_nf4_quantized_dq_amd as Q

    for v in (1e30, 1e-30, 1e-38):
        for t in (BF, F32):
            g = [torch.full((1000,), v, dtype=t, device="cuda")]
            norm = Q.grad_norm(Q.GradList(g))
            torch.cuda.synchronize()
            ref = T.grad_norm(_np(g))
            assert abs(float(norm) - ref) <= 2 * U * ref + 1e-45


def test_infinities_nan_zeros_and_limits(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    for bad in (float("inf"), -float("inf"), float("nan")):
        g = _tensors([100, 5000], [BF, F32], seed=2)
        g[1][4321] = bad
        gl = Q.GradList(g)
        norm = Q.grad_clip(gl, 1.0)
        torch.cuda.synchronize()
        if bad != bad:
            assert torch.isnan(norm).all() and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
        else:  # c = 0: everything 0, the infinity itself NaN
            assert torch.isinf(norm).all() and not g[0].any() and torch.isnan(g[1][4321])
            assert int((g[1] != 0).sum()) == 1
    z = [torch.zeros(77, device="cuda"), torch.zeros(0, device="cuda")]
    norm = Q.grad_clip(Q.GradList(z), 1.0)
    torch.cuda.synchronize()
    assert float(norm) == 0 and not z[0].any()
    empty = [torch.zeros(0, dtype=BF, device="cuda")]
    norm = Q.grad_clip(Q.GradList(empty), 1.0)
    torch.cuda.synchronize()
    assert float(norm) == 0
    g = _tensors([500], [F32], seed=3)
    norm = Q.grad_clip(Q.GradList(g), 0.0)
    torch.cuda.synchronize()
    assert float(norm) > 0 and not g[0].any()


def test_many_tensors_and_repeated_use(gpu_lib):
    """More tensors than one launch describes; the values change between calls; the same bits for
    the same values, also on another stream and in a graph."""
    import bit_nf4_quantized_dq_amd as Q

    sizes = [(37 * i) % 3001 + 1 for i in range(333)]
    g = _tensors(sizes, [BF if i % 3 else F32 for i in range(333)], seed=5, std=1.0)
    out = [torch.empty(n, dtype=BF, device="cuda") for n in sizes]
    gl = Q.GradList(g, out=out)
    ws = Q.new_workspace(gl._ws_bytes)
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        Q.grad_clip(gl, 1.0, norm=norm, ws=ws)
    for k in range(3):
        for t in g:
            t.mul_(1.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        first, kept = norm.clone(), [t.clone() for t in out]
        ref = T.grad_norm(_np(g))
        assert abs(float(first) - ref) <= 2 * U * ref
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = Q.grad_clip(gl, 1.0)
        torch.cuda.synchronize()
        assert torch.equal(first, again) and all(torch.equal(a, b) for a, b in zip(kept, out))
    assert int(ws[:524288].sum()) == 0, "the counter head stays zero"


HP = dict(lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


@pytest.mark.parametrize("n", [1, 3, 1027, 300_001])
def test_clipped_adamw(gpu_lib, n):
    import bit_nf4_quantized_dq_amd as Q

    master, m, v, grad = I.optimizer_state(40 + n, n)
    hp = {k: float(np.float32(x)) for k, x in HP.items()}
    d = [t.cuda() for t in (master, m, v, grad)]
    param = torch.empty(n, dtype=BF, device="cuda")
    norm = Q.grad_norm(Q.GradList([d[3]]))
    max_norm = float(np.float32(0.25)) * float(norm)
    Q.adamw_step_clipped(d[0], d[1], d[2], d[3], norm, max_norm, 7, param=param, **HP)
    torch.cuda.synchronize()
    c = T.clip_coefficient(float(norm), float(np.float32(max_norm)))
    g = c * grad.double().numpy()
    th0, m0, v0 = (t.double().numpy() for t in (master, m, v))
    b1, b2 = hp["beta1"], hp["beta2"]
    m1, v1 = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
    M = b1 * np.abs(m0) + (1 - b1) * np.abs(g)
    den = np.sqrt(v1 / (1 - b2**7)) + hp["eps"]
    ss = hp["lr"] / (1 - b1**7)
    step = ss * m1 / den
    th1 = th0 * (1 - hp["lr"] * hp["weight_decay"]) - step
    assert np.all(np.abs(d[1].double().cpu().numpy() - m1) <= 16 * U * M + 1e-40)
    assert np.all(np.abs(d[2].double().cpu().numpy() - v1) <= 24 * U * v1 + 1e-40)
    tol = 2.0**-21 * (2 * np.abs(th0) + 12 * np.abs(step) + 4 * ss * M / den)
    assert np.all(np.abs(d[0].double().cpu().numpy() - th1) <= tol)
    assert np.array_equal(param.view(torch.int16).cpu().numpy().view(np.uint16), O.bf16_round_bits(d[0].cpu().numpy()))


def test_clipped_adamw_below_the_limit_is_the_plain_step(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    n = 10_007
    state = I.optimizer_state(3, n)
    a, b = ([t.cuda() for t in state] for _ in range(2))
    norm = Q.grad_norm(Q.GradList([a[3]]))
    Q.adamw_step_clipped(a[0], a[1], a[2], a[3], norm, 1e6, 2, **HP)
    Q.adamw_step(b[0], b[1], b[2], b[3], 2, HP["lr"], weight_decay=HP["weight_decay"])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_clipped_adamw_skips_a_step_without_a_finite_norm(gpu_lib, bad):
    import bit_nf4_quantized_dq_amd as Q

    n = 5003
    state = [t.cuda() for t in I.optimizer_state(4, n)]
    state[3][100] = bad
    keep = [t.clone() for t in state]
    param = torch.full((n,), 3.0, dtype=BF, device="cuda")
    norm = Q.grad_norm(Q.GradList([state[3]]))
    Q.adamw_step_clipped(*state, norm, 1.0, 1, param=param, **HP)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(state[:3], keep[:3])) and torch.all(param == 3.0)
