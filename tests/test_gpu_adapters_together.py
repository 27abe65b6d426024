"""The adapters' operators together, as they are used: a training step of two adapted linears with
dropout on their inputs and on the residual branch (several adapters in one batch, clipped and
stepped by AdamW on flat buffers), and the serving of the trained adapters from the same memory."""

import pytest
import torch

from oracle import adapters_oracle as AO

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
SEED, P = 24680, 0.1
HALF = 2.0**-8


class Block:
    """z = x + drop(linear1(x)), y = linear2(z); n adapters on both linears, views of flat buffers."""

    def __init__(self, d, f, ranks, seed=0):
        import bit_nf4_quantized_dq_amd as Q

        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).cuda()  # noqa: E731
        self.shapes = [(d, d), (f, d)]
        self.q = [Q.quantize(rand(n, k, std=k**-0.5)) for n, k in self.shapes]
        init = []
        for n, k in self.shapes:
            init += [rand(r, k, std=k**-0.5) for r in ranks]
            # multiples of 1/64 up to 1/16, so that steps by 1/4 are exact in BF16
            init += [(torch.randint(-4, 5, (n, r), generator=gen) / 64).cuda() for r in ranks]
        # each tensor on a 16-byte boundary of the flat buffers
        sizes = [t.numel() for t in init]
        self.master = torch.cat([t.reshape(-1) for t in init])
        self.param, self.grad = self.master.to(BF16), torch.zeros_like(self.master, dtype=BF16)
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        cut = lambda flat: [p.view(t.shape) for p, t in zip(flat.split(sizes), init)]  # noqa: E731
        self.params, self.grads, n = cut(self.param), cut(self.grad), len(ranks)
        part = lambda ts, i: (ts[2 * n * i:2 * n * i + n], ts[2 * n * i + n:2 * n * (i + 1)])  # noqa: E731
        self.alpha = [16.0 + 8 * i for i in range(n)]
        self.sets = []
        for i in range(2):
            (A, B), (dA, dB) = part(self.params, i), part(self.grads, i)
            self.sets.append(Q.AdapterSet(A, B, self.alpha, dA=dA, dB=dB))
        # one generator state per use of dropout
        self.rng = [torch.tensor([SEED, i], device="cuda") for i in range(3)]

    def forward(self, x, ids, p):
        import bit_nf4_quantized_dq_amd as Q

        M = x.shape[0]
        T = [torch.empty(M, s.t_width, device="cuda") for s in self.sets]
        u = Q.linear_adapters_fwd(self.q[0], self.sets[0], x, ids, dropout=p, rng=self.rng[0], T_save=T[0])
        z = Q.dropout(u, p, self.rng[1], residual=x)
        y = Q.linear_adapters_fwd(self.q[1], self.sets[1], z, ids, dropout=p, rng=self.rng[2], T_save=T[1])
        return y, (u, z, T)

    def backward(self, x, ids, dy, saved, p):
        import bit_nf4_quantized_dq_amd as Q

        u, z, T = saved
        dz = Q.linear_adapters_bwd(self.q[1], self.sets[1], z, dy, ids, dropout=p, rng=self.rng[2], T_saved=T[1])
        du = Q.dropout(dz, p, self.rng[1])
        dx = Q.linear_adapters_bwd(self.q[0], self.sets[0], x, du, ids, dropout=p, rng=self.rng[0], T_saved=T[0])
        return dz, du, dx


def setup(M, seed=1):
    b = Block(256, 384, [16, 8, 40])
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, 256, generator=gen).cuda().to(BF16)
    dy = torch.randn(M, 384, generator=gen).cuda().to(BF16)
    ids = torch.randint(-1, 3, (M,), generator=gen).to(torch.int32).cuda()
    return b, x, dy, ids


@pytest.mark.parametrize("M", [24, 200])
@pytest.mark.parametrize("linear", [0, 1])
def test_gradient_is_the_slope(gpu_lib, M, linear):
    """sum(dy y) over a step of the linear's B along the sign of its gradient.  The chain is linear in
    B, so the change is <dB, step> but for the roundings to BF16 on the way, each at most half a
    step of its value: of y on both sides, of u and z (which reach the sum by |du| and |dz|, for
    linear 0), of dz and du (as much of the change of z and u), and of dB."""
    import bit_nf4_quantized_dq_amd as Q

    b, x, dy, ids = setup(M)
    y0, s0 = b.forward(x, ids, P)
    dz, du, _ = b.backward(x, ids, dy, s0, P)
    B, dB = b.sets[linear].B, [t.double() for t in b.sets[linear].dB]
    slope = 0.0
    for t, g in zip(B, dB):
        step = torch.sign(g) / 4
        slope += float((g * step).sum())
        moved = t.float() + step.float()
        t.copy_(moved)
        assert torch.equal(t.float(), moved)
    y1, s1 = b.forward(x, ids, P)
    d = lambda t: t.double()  # noqa: E731
    change = float((d(dy) * (d(y1) - d(y0))).sum())
    tol = HALF * float((d(dy).abs() * (d(y0).abs() + d(y1).abs())).sum()) + HALF * slope
    if linear == 0:
        (u0, z0, _), (u1, z1, _) = s0, s1
        tol += HALF * float((d(dz).abs() * (d(z0).abs() + d(z1).abs() + (d(z1) - d(z0)).abs())).sum())
        tol += HALF * float((d(du).abs() * (d(u0).abs() + d(u1).abs() + (d(u1) - d(u0)).abs())).sum())
    print(change, slope, tol, flush=True)
    assert tol < 0.5 * slope
    # second-order products of the roundings and the FP32 sums: a hundredth of the bound
    assert abs(change - slope) <= 1.01 * tol


def test_training_step_and_serving(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    M, lr, most = 200, 1e-2, 0.5
    b, x, dy, ids = setup(M)
    grads = Q.GradList(b.grads)
    for step in range(1, 3):
        before = b.master.clone()
        y, saved = b.forward(x, ids, P)
        dz, du, dx = b.backward(x, ids, dy, saved, P)
        # each linear's gradients, from the tensors that it was given
        for i, (inp, out) in enumerate(((x, du), (saved[1], dy))):
            s = b.sets[i]
            ref = AO.bwd(Q.dequantize(b.q[i]), s.A, s.B, b.alpha, inp, out, ids, P, (SEED, 2 * i), saved[2][i])
            for got, want, terms in zip(s.dA + s.dB, ref["dA"] + ref["dB"], ref["dA_sum"] + ref["dB_sum"]):
                assert ((got.double() - want).abs() <= HALF * want.abs() + 2.0**-12 * terms).all()
        raw = b.grad.double()
        norm = Q.grad_clip(grads, most)
        assert abs(float(norm) - float(raw.norm())) <= 2.0**-12 * float(norm) and float(norm) > most
        Q.adamw_step(b.master, b.m, b.v, b.grad, step, lr, param=b.param)
        moved = b.master - before
        assert torch.equal(b.param, b.master.to(BF16))
        # the first step of AdamW is lr against the gradient's sign
        if step == 1:
            big = b.grad.float().abs() > 1e-4
            assert big.any() and ((moved + lr * torch.sign(b.grad.float())).abs()[big] <= 1e-3 * lr).all()

    # the trained adapters serve from the same memory, in one batch with rows of the base alone
    A, B = b.sets[1].A, b.sets[1].B
    serve = Q.AdapterSet(A, B, b.alpha)
    z = saved[1]
    what = Q.dequantize(b.q[1])
    ref = AO.fwd(what, A, B, b.alpha, z, ids)
    tol = HALF * ref["Y"].abs() + 2.0**-13 * (ref["Y_base"] + ref["Y_branch"])
    for rows in (1, 2, 7, 64, M):
        got = Q.linear_adapters_fwd(b.q[1], serve, z[:rows], ids[:rows])
        assert ((got.double() - ref["Y"][:rows]).abs() <= tol[:rows]).all()
    base = ids < 0
    plain = Q.linear_adapters_fwd(b.q[1], serve, z, torch.full_like(ids, -1))
    got = Q.linear_adapters_fwd(b.q[1], serve, z, ids)
    assert torch.equal(got[base], plain[base]) and not torch.equal(got, plain)


def test_captured_training_steps(gpu_lib):
    """Forward, backward and clipping as one graph: its replays, on masks that differ, give the bits of
    eager calls, and an adapter that no row names gets zeros."""
    import bit_nf4_quantized_dq_amd as Q

    b, x, dy, ids = setup(96)
    ids[ids == 1] = 2
    grads = Q.GradList(b.grads)
    norm = torch.zeros(1, device="cuda")

    def step():
        y, saved = b.forward(x, ids, P)
        _, _, dx = b.backward(x, ids, dy, saved, P)
        Q.grad_clip(grads, 0.5, norm=norm)
        return y, dx

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.synchronize()
    for k in range(3):
        for i, r in enumerate(b.rng):
            r.copy_(torch.tensor([SEED + k, i]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, b.grad, norm)]
        want = (*step(), b.grad, norm)
        torch.cuda.synchronize()
        assert all(map(torch.equal, got, want)), k
        for s in b.sets:
            assert not s.dA[1].any() and not s.dB[1].any() and s.dA[0].any()
