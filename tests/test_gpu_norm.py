"""GPU parity of the block norms (qlora_norm_residual_fwd / bwd) against the FP64 oracle.

Tolerances, from the arithmetic.  u = 2^-24 is FP32's rounding; results in BF16 add one
rounding of relative 2^-8.
- A row's sum of d products: eight in a lane, then at most six adding steps in a wavefront and
  four across it, each one rounding of non-negative terms or relative to the terms' magnitude:
  20u.  1 / rms: half of that and four operations: 16u.
- Forward: q = y r_y w g is off by 20u |q|, x' by 24u (|s x| + |q|).  h = x' r_x w: relative
  20u, plus x's own error through x' and through r_x (relative rms(error) / rms(x')).
- Backward: the gradient t of x' sums terms of magnitude T (the oracle's), each off by at most
  80u: the factor k = r^3 mean(a x') carries three r (48u) and a sum (20u).  Products that
  follow add a few u; dy's correction is a difference of three sums with such factors (150u).
- Column sums add rows in segments and slices (at most 96 additions in a row of them here): 128u
  beside the terms' own error.
All together 256u of the oracle's magnitudes for every gradient, and the output's rounding."""

import os
import re

import numpy as np
import pytest
import torch

from oracle import training_oracle as T

pytestmark = pytest.mark.gpu
U, UB = 2.0**-24, 2.0**-8
BF, F32 = torch.bfloat16, torch.float32


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _case(M, d, stream, post, gate, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(1000 * M + 10 * d + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = dict(x=(2 * scale * r(M, d)).to(stream), y=(0.5 * scale * r(M, d)).to(BF), dh=(0.1 * r(M, d)).to(BF),
             dxo=(0.1 * r(M, d)).to(stream), w_post=(1 + 0.2 * r(d)).to(BF) if post else None, w_pre=(1 + 0.2 * r(d)).to(BF))
    rows = {"none": 0, "all": M, "each": 1}.get(gate, gate)
    c["gate"] = (0.5 + 0.3 * r(-(-M // rows), d)).to(BF) if rows else None
    return c, rows


def _cuda(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def _check_fwd(c, rows, post, s, eps, xo, h):
    n = {k: _np(v) for k, v in c.items()}
    args = (post, n["w_post"], n["gate"], rows, n["w_pre"], s, eps)
    x_ref, h_ref = T.norm_residual_fwd(n["x"], n["y"], *args)
    size = np.abs(s * n["x"])
    size = size + np.abs(x_ref - s * n["x"])
    e = 24 * U * size
    round_x = UB if c["x"].dtype == BF else U
    assert np.all(np.abs(_np(xo) - x_ref) <= e + round_x * (np.abs(x_ref) + e))
    if h is not None:
        r = 1 / np.sqrt(np.mean(x_ref**2, axis=1, keepdims=True) + eps)
        through_r = r * np.sqrt(np.mean(e**2, axis=1, keepdims=True))
        w = np.abs(n["w_pre"]) if n["w_pre"] is not None else 1.0
        tol = np.abs(h_ref) * (20 * U + through_r) + r * w * e
        assert np.all(np.abs(_np(h) - h_ref) <= tol + UB * (np.abs(h_ref) + tol))


def _check_bwd(c, rows, post, s, eps, got):
    n = {k: _np(v) for k, v in c.items()}
    ref, mag = T.norm_residual_bwd(n["x"], n["y"], n["dh"], n["dxo"], post, n["w_post"], n["gate"], rows, n["w_pre"], s,
                                   eps)
    stream = c["x"].dtype if c["x"] is not None else c["dxo"].dtype
    for name, t in zip(("dx", "dy", "dw_post", "dgate", "dw_pre"), got):
        if t is None:
            continue
        tol = 256 * U * mag[name]
        rnd = U if name == "dx" and stream == F32 else UB
        off = np.abs(_np(t) - ref[name])
        assert np.all(off <= tol + rnd * (np.abs(ref[name]) + tol) + 1e-37), (name, float(np.max(off)))


WIDTHS = [1, 3, 7, 8, 9, 15, 64, 511, 512, 513, 1000, 1025, 2047, 2051, 4096, 4097, 8191, 8192]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("stream", [BF, F32], ids=["bf16", "f32"])
def test_widths_and_rows(gpu_lib, d, stream):
    """Every workgroup size and row end, with one row and with several rows per workgroup."""
    import bit_nf4_quantized_dq_amd as Q

    for M, gate in ((1, "all"), (5, 2), (33, "each"), (70, "none")):
        print(f"norm M={M} d={d} gate={gate}", flush=True)
        c, rows = _case(M, d, stream, True, gate)
        g = _cuda(c)
        kw = dict(post_norm=True, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"], res_scale=0.9,
                  eps=1e-5)
        xo, h = Q.norm_residual_fwd(g["x"], g["y"], **kw)
        got = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
        torch.cuda.synchronize()
        _check_fwd(c, rows, True, np.float32(0.9), np.float32(1e-5), xo, h)
        _check_bwd(c, rows, True, np.float32(0.9), np.float32(1e-5), got)


@pytest.mark.parametrize("M,d,gate", [(2100, 513, 700), (2100, 96, "all"), (1500, 1000, 3), (1023, 2048, "each"),
                                      (999, 4096, 1000), (3000, 64, 7), (600, 8192, "all"), (2500, 1024, "none")])
def test_many_rows_and_gate_groups(gpu_lib, M, d, gate):
    """Segments inside a gate row's rows, of whole gate rows, and short last ones."""
    import bit_nf4_quantized_dq_amd as Q

    print(f"norm M={M} d={d} gate={gate}", flush=True)
    for post in (False, True):
        c, rows = _case(M, d, BF, post, gate)
        g = _cuda(c)
        kw = dict(post_norm=post, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"], eps=1e-6)
        xo, h = Q.norm_residual_fwd(g["x"], g["y"], **kw)
        got = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
        torch.cuda.synchronize()
        _check_fwd(c, rows, post, 1.0, np.float32(1e-6), xo, h)
        _check_bwd(c, rows, post, 1.0, np.float32(1e-6), got)


def test_large_operands_are_streamed_alike(gpu_lib):
    """Above 256 MB of operands the backward reads past the cache: same result as in two halves."""
    import bit_nf4_quantized_dq_amd as Q

    M, d = 4096, 6000
    print(f"norm M={M} d={d}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)  # noqa: E731
    x, y, dh, dxo, w1, w2 = r(M, d), r(M, d), r(M, d), r(M, d), r(d), r(d)
    kw = dict(post_norm=True, w_post=w1, w_pre=w2)
    dx, dy, dw1, _, dw2 = Q.norm_residual_bwd(x, y, dh, dxo, **kw)
    halves = [Q.norm_residual_bwd(x[i:i + 2048], y[i:i + 2048], dh[i:i + 2048], dxo[i:i + 2048], **kw) for i in (0, 2048)]
    torch.cuda.synchronize()
    assert torch.equal(dx, torch.cat([t[0] for t in halves])) and torch.equal(dy, torch.cat([t[1] for t in halves]))
    for got, k in ((dw1, 2), (dw2, 4)):
        both = halves[0][k].double() + halves[1][k].double()
        size = halves[0][k].double().abs() + halves[1][k].double().abs()
        # the halves and the whole are each rounded to BF16 once; sums of 4096 terms of magnitude 1
        assert torch.all((got.double() - both).abs() <= 2 * UB * size + 128 * U * 4096 * 8)


@pytest.mark.parametrize("have", ["norm only", "no next norm", "no block in the backward", "only dh", "only dx_out",
                                  "no weights"])
def test_operands_left_out(gpu_lib, have):
    import bit_nf4_quantized_dq_amd as Q

    M, d = 19, 200
    for stream in (BF, F32):
        c, rows = _case(M, d, stream, True, 4)
        kw = dict(post_norm=True, gate_rows=rows, res_scale=0.5, eps=1e-5)
        s, eps = 0.5, np.float32(1e-5)
        if have == "norm only":
            c.update(y=None, w_post=None, gate=None)
            g = _cuda(c)
            xo, h = Q.norm_residual_fwd(g["x"], w_pre=g["w_pre"], res_scale=0.5, eps=1e-5)
            torch.cuda.synchronize()
            _check_fwd(c, 0, False, s, eps, xo, h)
            continue
        if have == "no next norm":
            g = _cuda(c)
            xo, h = Q.norm_residual_fwd(g["x"], g["y"], pre_norm=False, w_post=g["w_post"], gate=g["gate"], **kw)
            torch.cuda.synchronize()
            assert h is None
            _check_fwd(dict(c), rows, True, s, eps, xo, None)
            continue
        if have == "no block in the backward":
            c.update(y=None, w_post=None, gate=None)
            kw.update(post_norm=False, gate_rows=0)
        elif have == "only dh":
            c.update(dxo=None)
        elif have == "only dx_out":
            c.update(dh=None, w_pre=None, x=None)
        elif have == "no weights":
            c.update(w_post=None, w_pre=None, gate=None)
        g = _cuda(c)
        more = dict(need_weights=False, need_gate=False) if have == "no weights" else {}
        got = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], w_post=g["w_post"], gate=g["gate"], w_pre=g["w_pre"],
                                  **kw, **more)
        torch.cuda.synchronize()
        assert (got[1] is None) == (c["y"] is None)
        _check_bwd(c, rows if c["gate"] is not None else 0, kw["post_norm"], s, eps, got)


def test_in_place(gpu_lib):
    """x_out over x and dx over dx_out give the same bits as separate outputs, also where the
    block has no norm of its own and where a row ends inside a lane's vector."""
    import bit_nf4_quantized_dq_amd as Q

    for d in (7, 200, 2051, 6001):
        for post in (False, True):
            for stream in (BF, F32):
                c, rows = _case(40, d, stream, post, "all")
                g = _cuda(c)
                kw = dict(post_norm=post, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"])
                for pre in (False, True):
                    xo, h = Q.norm_residual_fwd(g["x"], g["y"], pre_norm=pre, **{**kw, "w_pre": g["w_pre"] if pre else None})
                    x2 = g["x"].clone()
                    xo2, h2 = Q.norm_residual_fwd(x2, g["y"], pre_norm=pre, x_out=x2,
                                                  **{**kw, "w_pre": g["w_pre"] if pre else None})
                    torch.cuda.synchronize()
                    assert torch.equal(xo, xo2) and (not pre or torch.equal(h, h2)), (d, post, pre)
                a = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
                dxo2 = g["dxo"].clone()
                b = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], dxo2, dx=dxo2, **kw)
                torch.cuda.synchronize()
                assert all(p is q is None or torch.equal(p, q) for p, q in zip(a, b)), (d, post)


def test_special_rows(gpu_lib):
    """A row of zeros gives zeros (eps > 0); an infinity or NaN stays in its own row."""
    import bit_nf4_quantized_dq_amd as Q

    M, d = 12, 1001
    c, rows = _case(M, d, BF, True, "each")
    for k in ("x", "y"):
        c[k][3] = 0
    g = _cuda(c)
    kw = dict(post_norm=True, w_post=g["w_post"], gate=g["gate"], gate_rows=1, w_pre=g["w_pre"])
    clean = Q.norm_residual_fwd(g["x"], g["y"], **kw)
    back = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
    torch.cuda.synchronize()
    assert torch.all(clean[0][3] == 0) and torch.all(clean[1][3] == 0)
    _check_bwd(c, 1, True, 1.0, np.float32(1e-5), back)
    for bad in (float("nan"), float("inf")):
        x, y = g["x"].clone(), g["y"].clone()
        x[5, 1000] = bad
        y[8, 0] = bad
        xo, h = Q.norm_residual_fwd(x, y, **kw)
        dx, dy, _, _, _ = Q.norm_residual_bwd(x, y, g["dh"], g["dxo"], **kw)
        torch.cuda.synchronize()
        keep = [i for i in range(M) if i not in (5, 8)]
        assert torch.equal(xo[keep], clean[0][keep]) and torch.equal(h[keep], clean[1][keep])
        assert torch.equal(dx[keep], back[0][keep]) and torch.equal(dy[keep], back[1][keep])
        assert not torch.isfinite(xo[5, 1000]) and torch.isnan(h[5, 1000])


@pytest.mark.parametrize("M,d,rows", [(1, 700, 1), (1, 1280, 7), (1, 300, 7), (5, 1280, 5), (11, 700, 11), (11, 300, 4)])
@pytest.mark.parametrize("what", ["w_post", "gate"])
def test_infinite_weight_stays_in_its_sums(gpu_lib, what, M, d, rows):
    """An infinite post-norm weight or gate: the sum it multiplies is infinite in its column (over
    several rows the terms' signs may differ: not a number), and what does not pass through it is
    finite, for row counts that leave wavefronts without a row."""
    import bit_nf4_quantized_dq_amd as Q

    c, _ = _case(M, d, BF, True, rows)
    g = _cuda(c)
    g[what].view(-1)[d // 2] = float("inf")
    kw = dict(post_norm=True, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"])
    _, _, dw_post, dgate, dw_pre = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
    torch.cuda.synchronize()
    at = (slice(None), d // 2)
    hit, miss = (dgate, dw_post) if what == "w_post" else (dw_post, dgate)
    hit = hit.view(-1, d)
    assert torch.isinf(hit[at]).all() if M == 1 else not torch.isfinite(hit[at]).any()
    hit[at] = 0
    assert all(torch.isfinite(v).all() for v in (hit, miss, dw_pre))


def test_same_bits_again_on_another_stream_and_in_a_graph(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    M, d = 700, 1500
    c, rows = _case(M, d, BF, True, "all")
    g = _cuda(c)
    kw = dict(post_norm=True, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"])
    run = lambda **m: (*Q.norm_residual_fwd(g["x"], g["y"], **kw), *Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw, **m))  # noqa: E731
    a = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ws = Q.new_workspace(Q.norm_residual_workspace_size(M, d, rows))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(ws=ws)
    for k in range(3):
        g["x"].mul_(1.25)
        g["dh"].mul_(0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, eager)), k
    assert int(ws[:524288].sum()) == 0, "the counter head stays zero"


def test_slope_of_the_gpu_forward(gpu_lib):
    """The gradients against differences of the forward itself, in an FP32 stream: for
    L = <x', dx'> + <h, dh> summed in FP64, (L(x + e v) - L(x - e v)) / 2e against <dx, v>.  h is
    rounded to BF16: with e = 2^-4 each of the M d terms of <h, dh> is off by 2^-8 |h dh| at
    most, at random, so the difference quotient by about 2^-8 sqrt(M d) rms(h dh) / 2^-4; four
    times that, and e^2 of the second derivatives (below 1% of the slope's scale), are allowed."""
    import bit_nf4_quantized_dq_amd as Q

    M, d = 64, 512
    c, rows = _case(M, d, F32, True, "all")
    g = _cuda(c)
    kw = dict(post_norm=True, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"])
    v = torch.randn(M, d, generator=torch.Generator().manual_seed(9)).cuda()

    def L(x):
        xo, h = Q.norm_residual_fwd(x, g["y"], **kw)
        return float((xo.double() * g["dxo"].double()).sum() + (h.double() * g["dh"].double()).sum()), xo, h

    e = 2.0**-4
    slope = (L(g["x"] + e * v)[0] - L(g["x"] - e * v)[0]) / (2 * e)
    _, xo, h = L(g["x"])
    dx = Q.norm_residual_bwd(xo, g["y"], g["dh"], g["dxo"], **kw)[0]
    torch.cuda.synchronize()
    noise = 4 * UB * float((h.double() * g["dh"].double()).square().sum().sqrt()) / e
    scale = float(dx.double().square().sum().sqrt())
    assert abs(float((dx.double() * v.double()).sum()) - slope) <= noise + 0.01 * scale


@pytest.mark.parametrize("M,d", [(9, 5), (19, 200), (40, 2051)])
@pytest.mark.parametrize("scale,eps", [(1e15, 1e-5), (1e17, 0.0), (1e-14, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("stream", [BF, F32], ids=["bf16", "f32"])
def test_rows_of_any_magnitude(gpu_lib, M, d, scale, eps, stream):
    """Rows whose squares FP32 holds, whatever the cube of their norm: no gradient's term is lost or
    overflows, with and without a gradient from later blocks (which would hide small ones)."""
    import bit_nf4_quantized_dq_amd as Q

    print(f"norm M={M} d={d} scale={scale}", flush=True)
    for post in (True, False):
        c, rows = _case(M, d, stream, post, 4, scale=scale)
        for dxo in (c["dxo"], None):
            c["dxo"] = dxo
            g = _cuda(c)
            kw = dict(post_norm=post, w_post=g["w_post"], gate=g["gate"], gate_rows=rows, w_pre=g["w_pre"], eps=eps)
            xo, h = Q.norm_residual_fwd(g["x"], g["y"], **kw)
            got = Q.norm_residual_bwd(g["x"], g["y"], g["dh"], g["dxo"], **kw)
            torch.cuda.synchronize()
            _check_fwd(c, rows, post, 1.0, np.float32(eps), xo, h)
            _check_bwd(c, rows, post, 1.0, np.float32(eps), got)


def test_both_sides_of_the_cache_limit(gpu_lib):
    """Operands above a limit are read past the cache: one row more than fits below it gives the same
    bits for the other rows, and on both sides the column sums are the formula's in FP64."""
    import bit_nf4_quantized_dq_amd as Q

    source = os.path.join(os.path.dirname(Q.__file__), "csrc", "norm.hip")
    limit = int(re.search(r"> \(int64_t\)(\d+) << 20;", open(source).read()).group(1)) << 20
    d = 6000
    M = limit // (12 * d)  # BF16: four operands read, two written, of two bytes
    print(f"norm M={M}, {M + 1} d={d}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)  # noqa: E731
    x, y, dh, dxo, w1, w2 = r(M + 1, d), r(M + 1, d), r(M + 1, d), r(M + 1, d), r(d), r(d)
    D = lambda t: t.double()  # noqa: E731
    inv = lambda v: (v.square().mean(1, keepdim=True) + float(np.float32(1e-5))).rsqrt()  # noqa: E731
    u, a = D(x) * inv(D(x)), D(dh) * D(w2)
    t = D(dxo) + inv(D(x)) * (a - u * (a * u).mean(1, keepdim=True))
    t_abs = D(dxo).abs() + inv(D(x)) * (a.abs() + u.abs() * (a * u).abs().mean(1, keepdim=True))
    v = D(y) * inv(D(y))
    outs = []
    for m in (M, M + 1):
        got = Q.norm_residual_bwd(x[:m], y[:m], dh[:m], dxo[:m], post_norm=True, w_post=w1, w_pre=w2)
        torch.cuda.synchronize()
        outs.append(got)
        for k, terms, size in ((2, t * v, t_abs * v.abs()), (4, D(dh) * u, (D(dh) * u).abs())):
            want, tol = terms[:m].sum(0), 256 * U * size[:m].sum(0)
            assert torch.all((D(got[k]) - want).abs() <= tol + UB * (want.abs() + tol)), (m, k)
    assert torch.equal(outs[0][0], outs[1][0][:M]) and torch.equal(outs[0][1], outs[1][1][:M])
