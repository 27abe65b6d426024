"""Long reductions of the linear with many adapters, with tolerances that bind.  Rows of X (or of dY)
are zero but for a few columns, the first and the last ones among them: zeros add exactly, so
an element's sum has as many roundings as it has terms that are not zero, whatever the length.
Beside that the tolerances are test_gpu_adapters' own.  Each is also asserted to lie well below the
values that it is for."""

import pytest
import torch

from oracle import adapters_oracle as AO
from test_gpu_adapters import ADD, HALF, RNG, SPLIT

pytestmark = pytest.mark.gpu
FEW = 12


def sparse(gen, M, n):
    """[M, n] BF16: FEW values a row, in the first and last columns and spread over the rest."""
    at = torch.randint(0, n, (M, FEW), generator=gen, device="cuda")
    at[:, 0], at[:, 1] = 0, n - 1
    at[:, 2] = n - 1 - torch.arange(M, device="cuda") % 64
    at[:, 3] = torch.arange(M, device="cuda") * (n // M)
    x = torch.zeros(M, n, dtype=torch.bfloat16, device="cuda")
    return x.scatter_(1, at, torch.randn(M, FEW, generator=gen, device="cuda").bfloat16())


def near(got, ref, tol, name, share=0.05):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[0].tolist(), float(got[bad][0]), float(ref[bad][0]), float(tol[bad][0]))
    # a twentieth of the values: a lost term or a wrong column cannot pass
    some = ref[ref != 0].abs()
    assert len(some) and float(tol[ref != 0].median()) < share * float(some.median()), name


# rows, d_out, d_in, ranks, dropout: long reductions of T and Y, then of dX and G
@pytest.mark.parametrize("M,N,K,ranks,p", [
    (1, 16, 2**20 + 64, [16, 5], 0.0), (3, 48, 2**20 + 64, [16, 5], 0.2), (40, 16, 2**20 + 64, [40, 8], 0.0), (100, 32, 2**20 + 64, [16, 8], 0.0),
    (260, 16, 2**20 + 64, [8, 16], 0.0), (70, 16, 2**22, [16, 8], 0.0), (270, 16, 2**22, [24, 3], 0.0), (140, 1024, 2**22, [8, 16], 0.0),
    (1, 2**20 + 16, 64, [16, 5], 0.2), (40, 2**20 + 16, 64, [16, 5], 0.2), (100, 2**20 + 16, 64, [8, 40], 0.0), (260, 2**20 + 16, 64, [16, 5], 0.2),
    (70, 2**22, 64, [16, 8], 0.0), (270, 2**22, 64, [24, 3], 0.0), (140, 2**22, 1024, [8, 16], 0.0),
])
def test_long_reductions(gpu_lib, M, N, K, ranks, p):
    import bit_nf4_quantized_dq_amd as Q

    print(M, N, K, ranks, p, flush=True)
    gen = torch.Generator(device="cuda").manual_seed(M)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    long_in = K > N
    q = Q.quantize(randn(N, K))
    A, B = [randn(r, K).bfloat16() for r in ranks], [randn(N, r).bfloat16() for r in ranks]
    alpha = [float(r) for r in ranks]
    X = sparse(gen, M, K) if long_in else randn(M, K).bfloat16()
    dY = randn(M, N).bfloat16() if long_in else sparse(gen, M, N)
    ids = torch.randint(-1, len(ranks), (M,), generator=gen, device="cuda", dtype=torch.int32)
    ids[0] = 0
    s = Q.AdapterSet(A, B, alpha, dA=[torch.empty_like(t) for t in A], dB=[torch.empty_like(t) for t in B])
    kw = dict(dropout=p, rng=torch.tensor(RNG, device="cuda") if p else None)
    T = torch.empty(M, s.t_width, device="cuda")
    Y = Q.linear_adapters_fwd(q, s, X, ids, T_save=T, **kw)
    what = Q.dequantize(q)
    k, n, r = (FEW, N, s.t_width) if long_in else (K, FEW, s.t_width)
    ref = AO.fwd(what, A, B, alpha, X, ids, p, RNG)
    near(T, ref["T"], 2.0**-23 * ref["T"].abs() + ADD * (k + 8) * ref["T_sum"], "T")
    near(Y, ref["Y"], HALF * ref["Y"].abs() + ADD * (k + 8) * ref["Y_base"] + (ADD * (k + r + 16) + SPLIT) * ref["Y_branch"], "Y")
    del ref, Y
    dX = Q.linear_adapters_bwd(q, s, X, dY, ids, **kw)
    ref = AO.bwd(what, A, B, alpha, X, dY, ids, p, RNG)
    near(dX, ref["dX"], HALF * ref["dX"].abs() + ADD * (n + 8) * ref["dX_base"] + (ADD * (n + r + 16) + SPLIT) * ref["dX_branch"], "dX")
    for i in range(len(ranks)):
        if not (ids == i).any():
            assert not s.dA[i].any() and not s.dB[i].any()
            continue
        near(s.dA[i], ref["dA"][i], HALF * ref["dA"][i].abs() + (ADD * (n + M + 16) + SPLIT) * ref["dA_sum"][i], f"dA[{i}]")
        near(s.dB[i], ref["dB"][i], HALF * ref["dB"][i].abs() + (ADD * (k + M + 16) + SPLIT) * ref["dB_sum"][i], f"dB[{i}]")
    dA, dB = [t.clone() for t in s.dA], [t.clone() for t in s.dB]
    assert torch.equal(dX, Q.linear_adapters_bwd(q, s, X, dY, ids, **kw))
    assert all(map(torch.equal, dA + dB, s.dA + s.dB))


def test_as_many_adapters_as_a_set_holds(gpu_lib):
    """4096 adapters of two ranks, rows that name some of them in no order, and gradients of them all."""
    import bit_nf4_quantized_dq_amd as Q

    M, N, K, n = 700, 64, 128, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q = Q.quantize(randn(N, K))
    ranks = [8 if i % 3 else 70 for i in range(n)]
    A, B = [randn(r, K).bfloat16() for r in ranks], [randn(N, r).bfloat16() for r in ranks]
    s = Q.AdapterSet(A, B, 8.0, dA=[torch.full_like(t, 3.0) for t in A], dB=[torch.full_like(t, 3.0) for t in B])
    X, dY = randn(M, K).bfloat16(), randn(M, N).bfloat16()
    for rows in (1, 40, M):
        ids = torch.randint(-1, n, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        ids[0] = n - 1
        Y = Q.linear_adapters_fwd(q, s, X[:rows], ids)
        dX = Q.linear_adapters_bwd(q, s, X[:rows], dY[:rows], ids)
        named = sorted(set(ids.tolist()) - {-1})
        at = {a: i for i, a in enumerate(named)}
        few = torch.tensor([at.get(a, -1) for a in ids.tolist()], device="cuda")
        args = (Q.dequantize(q), [A[a] for a in named], [B[a] for a in named], [8.0] * len(named), X[:rows])
        f, b = AO.fwd(*args, few), AO.bwd(*args, dY[:rows], few)
        r = s.t_width
        near(Y, f["Y"], HALF * f["Y"].abs() + ADD * (K + 8) * f["Y_base"] + (ADD * (K + r + 16) + SPLIT) * f["Y_branch"], "Y")
        near(dX, b["dX"], HALF * b["dX"].abs() + ADD * (N + 8) * b["dX_base"] + (ADD * (N + r + 16) + SPLIT) * b["dX_branch"], "dX")
        for i, a in enumerate(named):
            near(s.dA[a], b["dA"][i], HALF * b["dA"][i].abs() + (ADD * (N + rows + 16) + SPLIT) * b["dA_sum"][i], f"dA[{a}]")
            near(s.dB[a], b["dB"][i], HALF * b["dB"][i].abs() + (ADD * (K + rows + 16) + SPLIT) * b["dB_sum"][i], f"dB[{a}]")
        none = sorted(set(range(n)) - set(named))
        assert not torch.cat([t.view(-1) for a in none for t in (s.dA[a], s.dB[a])]).any()


def kept_rows(rows, K, p):
    """[len(rows), K] bool: which elements of those rows of X stay (element m K + k has half e % 8 of block e // 8)."""
    import numpy as np

    block = (np.asarray(rows, dtype=np.uint64)[:, None] * np.uint64(K // 8) + np.arange(K // 8, dtype=np.uint64)).reshape(-1)
    low = np.uint64(0xFFFFFFFF)
    seed, offset = RNG
    ctr = np.stack([block & low, block >> np.uint64(32), np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)], 1)
    w = AO.philox(ctr, (seed & 0xFFFFFFFF, seed >> 32))
    return torch.from_numpy((np.stack([w & 0xFFFF, w >> 16], 2).reshape(len(rows), K) >= AO.threshold(p))).cuda()


@pytest.mark.parametrize("N,K", [(64, 8192), (8192, 64)])
def test_more_than_4_gib_of_rows(gpu_lib, N, K):
    """X, or dY, past 2^32 bytes, with dropout: rows at the start, at the 4 GiB mark and at the end.  (Dense
    rows: the bounds reach a twelfth of the values, and what is asked is whether the right rows are read.)"""
    import bit_nf4_quantized_dq_amd as Q

    print(N, K, flush=True)
    M, p, ranks = 2**18 + 4099, 0.1, [16, 5, 24]
    gen = torch.Generator(device="cuda").manual_seed(N)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q = Q.quantize(randn(N, K))
    A, B = [(randn(r, K) / 8).bfloat16() for r in ranks], [(randn(N, r) / 8).bfloat16() for r in ranks]
    s = Q.AdapterSet(A, B, [float(r) for r in ranks], dA=[torch.empty_like(t) for t in A], dB=[torch.empty_like(t) for t in B])
    X, dY = [torch.empty(M, n, dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for n in (K, N)]
    ids = torch.randint(-1, 3, (M,), generator=gen, device="cuda", dtype=torch.int32)
    rows = torch.tensor([*range(20), *range(2**18 - 10, 2**18 + 10), *range(M - 20, M)], device="cuda")
    kw = dict(dropout=p, rng=torch.tensor(RNG, device="cuda"))
    T = torch.empty(M, s.t_width, device="cuda")
    Y = Q.linear_adapters_fwd(q, s, X, ids, T_save=T, **kw)
    what, keep = Q.dequantize(q).double(), kept_rows(rows.tolist(), K, p)
    gate = keep.double() * AO.scale(p)
    x, dy, own = X[rows].double(), dY[rows].double(), ids[rows]
    # each row's own adapter, zeros for none
    wide = lambda ts, dim: torch.stack([torch.nn.functional.pad(t.double(), (0, 0, 0, 24 - t.shape[0]) if dim == 0 else (0, 24 - t.shape[1])) for t in ts])  # noqa: E731
    has = (own >= 0).double()
    Ar, Br = wide(A, 0)[own.clamp(min=0).long()] * has[:, None, None], wide(B, 1)[own.clamp(min=0).long()] * has[:, None, None]
    dot = lambda a, b: (a * b).sum(-1)  # noqa: E731
    xd = x * gate
    t, tm = dot(Ar, xd[:, None]), dot(Ar.abs(), xd.abs()[:, None])
    near(T[rows], t, 2.0**-23 * t.abs() + ADD * (K + 8) * tm, "T", 0.25)
    y, base = x @ what.T + dot(Br, t[:, None]), x.abs() @ what.abs().T
    near(Y[rows], y, HALF * y.abs() + ADD * (K + 8) * base + (ADD * (K + 40) + SPLIT) * dot(Br.abs(), tm[:, None]), "Y", 0.25)
    del Y
    dX = Q.linear_adapters_bwd(q, s, X, dY, ids, T_saved=T, **kw)
    g, gm = (dy[:, :, None] * Br).sum(1), (dy.abs()[:, :, None] * Br.abs()).sum(1)
    back, backm = (g[:, :, None] * Ar).sum(1) * gate, (gm[:, :, None] * Ar.abs()).sum(1) * gate
    ref = dy @ what + back
    near(dX[rows], ref, HALF * ref.abs() + ADD * (N + 8) * (dy.abs() @ what.abs()) + (ADD * (N + 40) + SPLIT) * backm, "dX", 0.25)
    del dX
    # the gradients of those rows alone, few values each, by the T that was checked
    dy = sparse(gen, len(rows), N)
    dY.zero_()[rows] = dy
    assert Q.linear_adapters_bwd(q, s, X, dY, ids, T_saved=T, need_dx=False, **kw) is None
    dy, t = dy.double(), T[rows].double()
    g, gm = (dy[:, :, None] * Br).sum(1), (dy.abs()[:, :, None] * Br.abs()).sum(1)
    for i, r in enumerate(ranks):
        at = own == i
        assert at.any()
        dA, dAm = g[at, :r].T @ xd[at], gm[at, :r].T @ xd[at].abs()
        near(s.dA[i], dA, HALF * dA.abs() + (ADD * (FEW + 80) + SPLIT) * dAm, f"dA[{i}]")
        dB, dBm = dy[at].T @ t[at, :r], dy[at].abs().T @ t[at, :r].abs()
        near(s.dB[i], dB, HALF * dB.abs() + (ADD * 80 + SPLIT) * dBm, f"dB[{i}]")
