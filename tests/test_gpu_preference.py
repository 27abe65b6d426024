"""GPU parity of the token log-probabilities and the preference loss against the FP64 oracle.

Tolerances, from the arithmetic (u = 2^-24).  The sum of a row's exponentials adds V / threads
terms in a lane (at most 128 between rescalings of the sizes here), then some twelve merges;
each exponential is off by 2u and by its argument's rounding, 1.5u of the distance to the
maximum, weighted by its probability (at most log V on average): together below 200u relative,
which is the absolute error of the log-probability; its result is rounded to FP32 once.  Log
ratios add such errors (in FP64) and are rounded once.  A pair's slope changes by at most
beta^2 / 4P times the log ratios' error; a probability far from the maximum is off by 4u of the
distance more.  Gradients in BF16 add a rounding of 2^-8."""

import numpy as np
import pytest
import torch

from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
U, UB = 2.0**-24, 2.0**-8
BF, F32 = torch.bfloat16, torch.float32
LP = 200 * U


def _case(P, S, V, dtype, seed=0, masked=0.3):
    g = torch.Generator().manual_seed(P * 100003 + S * 1009 + V + seed)
    x = (2.5 * torch.randn(2 * P, S, V, generator=g)).to(dtype)
    labels = torch.randint(0, V, (2 * P, S), generator=g)
    labels[torch.rand(2 * P, S, generator=g) < masked] = -100
    ref = -torch.rand(2 * P, S, generator=g) * 5
    return x, labels, ref


def _check(x, labels, ref, beta, smoothing, scale, out, grad=True):
    loss, ratios, logps, d = out
    n, S, V = x.shape
    P = n // 2
    xn = x.double().numpy()
    loss_r, D, lp_r, d_r, c = T.preference_loss(xn, labels.numpy(), None if ref is None else ref.numpy(), beta, smoothing,
                                                scale)
    counted = ((labels >= 0) & (labels < V)).numpy()
    lp, D_g = logps.double().cpu().numpy(), ratios.double().cpu().numpy()
    assert np.all(np.abs(lp - lp_r) <= LP + U * np.abs(lp_r)) and np.all(lp[~counted] == 0)
    tol_D = LP * counted.sum(axis=1)
    assert np.all(np.abs(D_g - D) <= tol_D + U * np.abs(D))
    tol_z = np.abs(beta) * (tol_D[:P] + tol_D[P:])
    assert abs(float(loss) - loss_r) <= tol_z.mean() + 4 * U * abs(loss_r)
    if not grad:
        assert d is None
        return
    dg = d.double().cpu().numpy()
    m = xn.max(axis=2, keepdims=True)
    p = np.exp(xn - m) / np.exp(xn - m).sum(axis=2, keepdims=True)
    hot = np.zeros_like(p)
    idx = np.where(counted, labels.numpy(), 0)
    np.put_along_axis(hot, idx[..., None], 1.0, axis=2)
    dc = abs(scale * beta) / P * 0.25 * np.concatenate([tol_z, tol_z])[:, None, None]
    far = np.where(p > 0, np.abs(xn - m), 0.0)  # (-inf has probability 0)
    tol = np.abs(c)[:, None, None] * (p * (LP + 4 * U * far) + 4 * U * hot) + (dc + 2 * U * np.abs(c)[:, None, None]) * np.abs(hot - p)
    rnd = UB if x.dtype == BF else U
    ok = np.abs(dg - d_r) <= tol + rnd * np.abs(d_r) + 1e-37
    assert np.all(ok[counted]) and np.all(dg[~counted] == 0)


@pytest.mark.parametrize("P,S,V", [(1, 1, 1), (1, 1, 2), (2, 3, 7), (1, 5, 8), (3, 4, 9), (1, 33, 1003), (2, 17, 8192),
                                   (2, 9, 8193), (1, 7, 16385), (1, 2, 70001), (5, 11, 513)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_sizes(gpu_lib, P, S, V, dtype):
    """Odd vocabularies, rows that are split over workgroups (few rows, wide ones), one token."""
    import bit_nf4_quantized_dq_amd as Q

    print(f"preference P={P} S={S} V={V}", flush=True)
    x, labels, ref = _case(P, S, V, dtype)
    for smoothing, r in ((0.0, ref), (0.25, None)):
        out = Q.preference_loss(x.cuda(), labels.cuda(), None if r is None else r.cuda(), 0.5, smoothing, 2.0)
        lp = Q.token_logps(x.cuda(), labels.cuda())
        torch.cuda.synchronize()
        _check(x, labels, r, 0.5, float(np.float32(smoothing)), 2.0, out)
        assert torch.equal(lp, out[2])


@pytest.mark.parametrize("V", [33000, 66000, 131072, 140000])
def test_wide_rows_in_whole(gpu_lib, V):
    """Many rows are not split: every workgroup size, and the elements after the batches."""
    import bit_nf4_quantized_dq_amd as Q

    P, S = 2, 256
    print(f"preference V={V}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = (2.5 * torch.randn(2 * P, S, V, generator=gen, device="cuda")).to(BF)
    labels = torch.full((2 * P, S), -100, device="cuda")
    rows = [(0, 0), (0, 255), (1, 7), (2, 100), (3, 254)]
    for i, (a, b) in enumerate(rows):
        labels[a, b] = (V - 1) * i // 4
    out = Q.preference_loss(x, labels, None, 0.1)
    torch.cuda.synchronize()
    xs = x.cpu()
    keep = torch.stack([xs[a, b] for a, b in rows])
    lp = T.token_logps(keep.double().numpy(), np.array([int(labels[a, b]) for a, b in rows]))
    got = np.array([float(out[2][a, b]) for a, b in rows])
    assert np.all(np.abs(got - lp) <= LP + U * np.abs(lp))
    D = np.array([lp[0] + lp[1], lp[2], lp[3], lp[4]])
    z = 0.1 * (D[:2] - D[2:])
    c = 0.05 * (1 / (1 + np.exp(-z)) - 1)
    c = np.concatenate([c, -c])
    for k, (a, b) in enumerate(rows):
        xk = keep[k].double().numpy()
        p = np.exp(xk - xk.max())
        p /= p.sum()
        want = -c[a] * p
        want[int(labels[a, b])] += c[a]
        off = np.abs(out[3][a, b].double().cpu().numpy() - want)
        assert np.all(off <= abs(c[a]) * (p * (LP + 4 * U * (xk.max() - xk)) + 1e-6) + UB * np.abs(want))
    assert int((out[3].view(torch.int16)[labels < 0] != 0).sum()) == 0


def test_masks(gpu_lib):
    """All tokens of an answer masked, of a pair, of the batch; labels outside the vocabulary on
    either side; what stands in masked rows is not read (NaN)."""
    import bit_nf4_quantized_dq_amd as Q

    P, S, V = 3, 6, 600
    for dtype in (BF, F32):
        x, labels, ref = _case(P, S, V, dtype, masked=0.2)
        labels[1] = -100             # a chosen answer
        labels[2] = V                # a pair: chosen ...
        labels[5] = 1 << 40          # ... and rejected
        labels[0, 0] = -1
        labels[3, 5] = -(1 << 62)
        clean = x.clone()
        gone = (labels < 0) | (labels >= V)
        x[gone] = float("nan")
        ref[gone] = float("nan")
        out = Q.preference_loss(x.cuda(), labels.cuda(), ref.cuda(), 0.3)
        torch.cuda.synchronize()
        _check(clean, labels, torch.where(gone, torch.zeros_like(ref), ref), 0.3, 0.0, 1.0, out)
        labels[:] = -100
        out = Q.preference_loss(x.cuda(), labels.cuda(), ref.cuda(), 0.3)
        torch.cuda.synchronize()
        assert abs(float(out[0]) - np.log(2)) <= U and not out[1].any() and not out[2].any() and not out[3].any()


@pytest.mark.parametrize("V,split", [(600, False), (20000, True), (40000, False)])
def test_masked_vocabulary_and_extremes(gpu_lib, V, split):
    """Vocabulary entries at -inf or the type's lowest value have probability 0; a row that is the
    lowest value throughout is uniform; very large logits; +inf, NaN and a row of -inf give NaN."""
    import bit_nf4_quantized_dq_amd as Q

    rows = 16 if split else 1024
    for dtype in (BF, F32):
        gen = torch.Generator().manual_seed(V)
        x = (2 * torch.randn(rows, V, generator=gen)).to(dtype)
        low = torch.finfo(dtype).min
        labels = torch.full((rows,), -100)
        labels[:10] = torch.tensor([0, 5, V - 1, 17, 3, 4, V // 2, 9, 1, 2])
        x[0, 8:] = -float("inf")              # most of the row, whole workgroup parts among it
        x[1, : V - 4] = low
        x[1, 5] = 1.0
        x[2, : V - 1] = -float("inf")         # only the label is left
        x[3] = low                            # nothing is left: uniform
        x[4] = 3e38
        x[5] = -2e30
        x[5, 4] = -2e30 * 1.01
        x[6, 100] = 2e38
        x[7, 11] = float("inf")
        x[8, 11] = float("nan")
        x[9] = -float("inf")
        lp = Q.token_logps(x.cuda(), labels.cuda()).double().cpu().numpy()
        torch.cuda.synchronize()
        xn = x[:7].double().numpy()
        ref = T.token_logps(xn, labels[:7].numpy())
        assert np.all(np.abs(lp[:7] - ref) <= LP + 2 * U * np.abs(ref)), (dtype, lp[:7], ref)
        assert np.all(np.isnan(lp[7:10])) and np.all(lp[10:] == 0)


def test_gradient_under_masked_vocabulary(gpu_lib):
    """Entries of probability 0 get a gradient of 0, also where most of a row is -inf or the type's
    lowest value; a row that is the lowest value throughout is uniform."""
    import bit_nf4_quantized_dq_amd as Q

    for V in (300, 9001):
        for dtype in (BF, F32):
            x, labels, ref = _case(1, 4, V, dtype, masked=0.0)
            low = torch.finfo(dtype).min
            x[0, 0, 7:] = -float("inf")
            labels[0, 0] = 3
            x[0, 1, : V - 2] = low
            labels[0, 1] = V - 1
            x[1, 2] = low
            x[1, 3, ::2] = low
            labels[1, 3] = 1
            out = Q.preference_loss(x.cuda(), labels.cuda(), ref.cuda(), 0.25)
            torch.cuda.synchronize()
            _check(x, labels, ref, 0.25, 0.0, 1.0, out)
            d = out[3].float().cpu()
            assert not d[0, 0, 7:].any() and not d[0, 1, : V - 2].any() and not d[1, 3, ::2].any()


def test_infinite_differences(gpu_lib):
    """A label of probability 0: the loss is infinite for a chosen answer, 0 for a rejected one, and
    the gradient stays finite."""
    import bit_nf4_quantized_dq_amd as Q

    x, labels, ref = _case(1, 3, 50, F32, masked=0.0)
    for side, want in ((0, float("inf")), (1, 0.0)):
        y = x.clone()
        y[side, 1, labels[side, 1]] = -float("inf")
        loss, ratios, lp, d = Q.preference_loss(y.cuda(), labels.cuda(), ref.cuda(), 0.1)
        torch.cuda.synchronize()
        assert float(loss) == want and float(ratios[side]) == -float("inf") and torch.isfinite(d).all()
    y = x.clone()
    y[0, 1, labels[0, 1]] = -float("inf")
    loss = Q.preference_loss(y.cuda(), labels.cuda(), ref.cuda(), 0.1, label_smoothing=0.1)[0]
    torch.cuda.synchronize()
    assert float(loss) == float("inf")


def test_in_place_and_loss_alone(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    for P, S, V, dtype in ((2, 5, 1003, BF), (1, 2, 40001, F32), (1, 600, 77, BF), (1, 3, 5, F32)):
        x, labels, ref = _case(P, S, V, dtype)
        xd, ld, rd = x.cuda(), labels.cuda(), ref.cuda()
        a = Q.preference_loss(xd, ld, rd, 0.2)
        alone = Q.preference_loss(xd, ld, rd, 0.2, need_grad=False)
        y = xd.clone()
        b = Q.preference_loss(y, ld, rd, 0.2, dlogits=y)
        torch.cuda.synchronize()
        assert b[3] is y and all(torch.equal(p, q) for p, q in zip(a, b))
        assert alone[3] is None and all(torch.equal(p, q) for p, q in zip(a[:3], alone[:3]))
        _check(x, labels, ref, float(np.float32(0.2)), 0.0, 1.0, a)


def test_beyond_32_bit_offsets(gpu_lib):
    """The last rows of 2.3 * 2^31 logits (9.9 GB in BF16), and their gradients in place."""
    import bit_nf4_quantized_dq_amd as Q

    S, V = 18841, 131072
    print("preference over 4.9e9 logits", flush=True)
    x = torch.zeros(2, S, V, dtype=BF, device="cuda")
    labels = torch.full((2, S), -100, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows = [(0, 0), (0, 16500), (1, 3), (1, S - 1)]
    keep = []
    for a, b in rows:
        x[a, b] = (2 * torch.randn(V, generator=gen, device="cuda")).to(BF)
        labels[a, b] = 131 * (b % 1000)
        keep.append(x[a, b].double().cpu().numpy())
    lp = T.token_logps(np.stack(keep), np.array([int(labels[a, b]) for a, b in rows]))
    loss, D, lps, d = Q.preference_loss(x, labels, None, 0.1, dlogits=x)
    torch.cuda.synchronize()
    got = np.array([float(lps[a, b]) for a, b in rows])
    assert np.all(np.abs(got - lp) <= LP + U * np.abs(lp))
    z = 0.1 * (lp[0] + lp[1] - lp[2] - lp[3])
    c = 0.1 * (1 / (1 + np.exp(-z)) - 1)
    for k, (a, b) in enumerate(rows):
        p = np.exp(keep[k] - keep[k].max())
        p /= p.sum()
        want = -(c if a == 0 else -c) * p
        want[int(labels[a, b])] += c if a == 0 else -c
        assert np.all(np.abs(d[a, b].double().cpu().numpy() - want) <= abs(c) * (p * 1e-4 + 1e-6) + UB * np.abs(want))
    del x, d
    torch.cuda.empty_cache()


def test_same_bits_again_on_another_stream_and_in_a_graph(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    P, S, V = 3, 40, 9000
    x, labels, ref = (t.cuda() for t in _case(P, S, V, BF))
    a = Q.preference_loss(x, labels, ref, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = Q.preference_loss(x, labels, ref, 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ws = Q.new_workspace(Q.preference_workspace_size(P, S, V))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = Q.preference_loss(x, labels, ref, 0.1, ws=ws)
    for k in range(4):
        x.mul_(0.9)
        labels.copy_(labels.roll(1, 1))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = Q.preference_loss(x, labels, ref, 0.1)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, eager)), k
    assert int(ws[:524288].sum()) == 0, "the counter head stays zero"


def test_slope_of_the_gpu_loss(gpu_lib):
    """The gradient against differences of the loss itself (FP32 logits): the step e = 2^-3 along a
    random direction changes the loss by e |slope|; its rounding (4u of the loss over 2e) and e^2 of
    the third derivatives, below 2% of the gradient's norm, are allowed."""
    import bit_nf4_quantized_dq_amd as Q

    x, labels, ref = (t.cuda() for t in _case(2, 8, 300, F32, masked=0.1))
    v = torch.randn(x.shape, generator=torch.Generator().manual_seed(4)).cuda()
    v /= v.norm()
    f = lambda t: float(Q.preference_loss(t, labels, ref, 0.3, need_grad=False)[0])  # noqa: E731
    d = Q.preference_loss(x, labels, ref, 0.3)[3]
    e = 2.0**-3
    slope = (f(x + e * v) - f(x - e * v)) / (2 * e)
    torch.cuda.synchronize()
    assert abs(float((d.double() * v.double()).sum()) - slope) <= 4 * U * 5 / (2 * e) + 0.02 * float(d.norm())


MASKS = (-1e9, -5e9, -1e10, -1e20, -1e29, -1e30)
TOPS = (5e9, 1e10, 1e20)
BASES = tuple(s * b for b in (2e6, 2.0**21, 2.0**22 - 1, 2.0**22, 2.0**22 + 1, 2.0**23, 1e7, 3e9) for s in (1, -1))


def _finite_masks(V, gen):
    """Rows of finite logits of any magnitude, and a label for each: entries masked by a large
    negative number in the first columns, all but four, every second one, or all; one entry far
    above the others; whole rows far from zero, in steps of one and in stripes of eight columns
    that differ by three (neighbouring threads' vectors)."""
    rows, labels = [], []

    def add(x, label):
        rows.append(x)
        labels.append(int(label))

    for k, v in enumerate(MASKS):
        few = torch.randperm(V, generator=gen)[:4]
        keeps = (torch.arange(V) >= V - 4, torch.zeros(V, dtype=torch.bool).index_fill(0, few, True),
                 torch.arange(V) % 2 == 1, torch.zeros(V, dtype=torch.bool))
        for keep in keeps:
            x = torch.where(keep, 2 * torch.randn(V, generator=gen), torch.full((V,), v))
            left = keep.nonzero()[:, 0]
            add(x, left[k % len(left)] if len(left) else V // 2)
        add(rows[-4], 1)  # a label that is masked
    for v in TOPS:
        x = 2 * torch.randn(V, generator=gen)
        x[V // 3] = v
        add(x, V // 3)
        add(x, 7)
    for b in BASES:
        add(b + torch.randint(-6, 7, (V,), generator=gen).float(), V - 1)
        add(b + 1 - 3 * (torch.arange(V) // 8 % 2).float(), 3)
    return torch.stack(rows), torch.tensor(labels)


@pytest.mark.parametrize("rows,V", [(1024, 2051), (1024, 5000), (256, 40000), (256, 66000), (160, 140000), (100, 20000),
                                    (100, 140000)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_finite_logits_of_any_magnitude(gpu_lib, rows, V, dtype):
    """Finite logits give finite log-probabilities, for every workgroup size, whole rows and split
    ones (fewer than 128), and masks that leave most threads nothing."""
    import bit_nf4_quantized_dq_amd as Q

    print(f"token logps rows={rows} V={V}", flush=True)
    x, at = _finite_masks(V, torch.Generator().manual_seed(V))
    n = len(x)
    assert n <= rows
    x = torch.cat([x, torch.zeros(rows - n, V)]).to(dtype)
    labels = torch.cat([at, torch.full((rows - n,), -100)])
    lp = Q.token_logps(x.cuda(), labels.cuda()).double().cpu().numpy()
    torch.cuda.synchronize()
    ref = T.token_logps(x[:n].double().numpy(), at.numpy())
    bad = np.nonzero(~(np.abs(lp[:n] - ref) <= LP + 2 * U * np.abs(ref)))[0]
    assert len(bad) == 0, [(int(i), lp[i], ref[i]) for i in bad[:5]]
    assert np.all(lp[n:] == 0)


@pytest.mark.parametrize("S,V", [(3, 2051), (80, 2051), (80, 9001), (3, 20000)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradient_under_finite_masks(gpu_lib, S, V, dtype):
    """The same rows in a pair: loss and gradient, in place too (rows below 128 in all are split)."""
    import bit_nf4_quantized_dq_amd as Q

    print(f"preference S={S} V={V}", flush=True)
    rows, at = _finite_masks(V, torch.Generator().manual_seed(V + 1))
    top = rows.gather(1, at[:, None])[:, 0] >= rows.amax(1) - 30  # labels that are not masked away
    rows, at = rows[top], at[top]
    for first in range(0, len(rows), 2 * S):
        x, labels, ref = _case(1, S, V, F32, masked=0.2)
        take = rows[first:first + 2 * S]
        x.view(-1, V)[:len(take)] = take
        labels.view(-1)[:len(take)] = at[first:first + 2 * S]
        x = x.to(dtype)
        out = Q.preference_loss(x.cuda(), labels.cuda(), ref.cuda(), 0.25)
        y = x.cuda()
        place = Q.preference_loss(y, labels.cuda(), ref.cuda(), 0.25, dlogits=y)
        torch.cuda.synchronize()
        _check(x, labels, ref, 0.25, 0.0, 1.0, out)
        assert all(torch.equal(a, b) for a, b in zip(out, place))
