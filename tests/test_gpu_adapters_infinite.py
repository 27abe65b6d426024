"""Infinite operands of the linear with many adapters: infinities and NaN come out where the definition
has them (FP64 on the CPU), with their signs, and everything else is as near as ever.  Tolerances
as in test_gpu_adapters."""

import pytest
import torch

from oracle import adapters_oracle as AO
from test_gpu_adapters import ADD, HALF, RNG, SPLIT, make

pytestmark = pytest.mark.gpu
INF = float("inf")
CASES = [  # rows, d_out, d_in, ranks
    # T posted within the launch; T by a launch, one and two weight tiles to a workgroup
    (4, 1040, 320, [16, 8, 24]), (4, 1040, 320, [16, 5, 24]), (40, 272, 320, [16, 5, 24]), (61, 8192, 320, [24, 5, 8]), (100, 1024, 320, [24, 40, 8]),
    # tiles of 128 and 256 rows over the codes, whole and split
    (140, 272, 320, [16, 8, 24]), (140, 272, 320, [16, 5, 24]), (520, 6672, 128, [16, 20, 8]), (513, 128, 6720, [8, 64, 9]), (447, 208, 2112, [9, 40, 8]),
    # the decoded copy, for Y and for dX
    (1030, 5776, 64, [16, 20, 8]), (1030, 64, 5824, [8, 64, 24]),
]


def agree(got, ref, tol, name):
    got, ref, tol = got.double().cpu(), ref.cpu(), tol.cpu()
    assert torch.equal(got.isnan(), ref.isnan()), (name, int((got.isnan() != ref.isnan()).sum()), int(ref.isnan().sum()))
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf]) and not got[~inf].isinf().any(), name
    fin = ref.isfinite()
    assert ((got - ref).abs()[fin] <= tol[fin]).all(), name


def plant(c, what):
    """A few infinities; the first adapter's rows (0, 4, ...) hold the ones in X and dY."""
    A, B, X, dY = c["A"][0], c["B"][0], c["X"], c["dY"]
    if what == "B":
        B[3, 1], B[9, 0], B[10, 5] = INF, -INF, INF
    elif what == "A":
        A[1, 7], A[6, 20] = INF, -INF
    elif what == "X":
        X[0, 13], X[-1, 40] = INF, -INF
    elif what == "dY":
        dY[0, 11], dY[-1, 2] = -INF, INF


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("what", ["A", "B", "X", "dY"])
@pytest.mark.parametrize("shape", CASES)
def test_infinities_are_the_definitions(gpu_lib, shape, what, p):
    import bit_nf4_quantized_dq_amd as Q

    print(shape, what, p, flush=True)
    M, N, K, ranks = shape
    c = make(7, M, N, K, ranks, "tokens")
    c["ids"] = torch.arange(M, dtype=torch.int32, device="cuda") % 4
    c["ids"][c["ids"] == 3] = -1
    c["ids"][-1] = 0
    plant(c, what)
    r = c["set"].t_width
    T = torch.empty(M, r, device="cuda")
    Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=p, rng=c["rng"] if p else None, T_save=T)
    dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"], dropout=p, rng=c["rng"] if p else None)
    host = [c["what"].cpu(), [t.cpu() for t in c["A"]], [t.cpu() for t in c["B"]], c["alpha"], c["X"].cpu()]
    ids = c["ids"].cpu()
    f = AO.fwd(*host, ids, p, RNG)
    b = AO.bwd(*host, c["dY"].cpu(), ids, p, RNG)
    agree(T, f["T"], 2.0**-23 * f["T"].abs() + ADD * (K + 8) * f["T_sum"], "T")
    agree(Y, f["Y"], HALF * f["Y"].abs() + ADD * (K + 8) * f["Y_base"] + (ADD * (K + r + 16) + SPLIT) * f["Y_branch"], "Y")
    agree(dX, b["dX"], HALF * b["dX"].abs() + ADD * (N + 8) * b["dX_base"] + (ADD * (N + r + 16) + SPLIT) * b["dX_branch"], "dX")
    for i in range(len(ranks)):
        agree(c["set"].dA[i], b["dA"][i], HALF * b["dA"][i].abs() + (ADD * (N + M + 16) + SPLIT) * b["dA_sum"][i], f"dA[{i}]")
        agree(c["set"].dB[i], b["dB"][i], HALF * b["dB"][i].abs() + (ADD * (K + M + 16) + SPLIT) * b["dB_sum"][i], f"dB[{i}]")
    # the infinities came through
    assert any(t.isinf().any() for t in (f["Y"], b["dX"], *b["dA"], *b["dB"]))


@pytest.mark.parametrize("ranks", [[16, 8, 24], [16, 5, 24], [5, 16, 24]])
@pytest.mark.parametrize("M,N,K", [(4, 1040, 320), (40, 272, 320), (140, 272, 320), (700, 592, 128)])
def test_an_infinity_in_the_last_row_of_b(gpu_lib, M, N, K, ranks):
    """d_out past a multiple of 64: G = dY B takes nothing from beyond B's last row, whatever it holds
    and whatever ranks the set's other adapters have."""
    import bit_nf4_quantized_dq_amd as Q

    print(M, N, K, ranks, flush=True)
    c = make(9, M, N, K, ranks, "tokens")
    c["ids"] = torch.arange(M, dtype=torch.int32, device="cuda") % 3
    c["B"][0][-1, 2] = INF
    dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"])
    b = AO.bwd(c["what"].cpu(), [t.cpu() for t in c["A"]], [t.cpu() for t in c["B"]], c["alpha"], c["X"].cpu(), c["dY"].cpu(), c["ids"].cpu())
    r = c["set"].t_width
    assert b["dX"].isinf().any()
    agree(dX, b["dX"], HALF * b["dX"].abs() + ADD * (N + 8) * b["dX_base"] + (ADD * (N + r + 16) + SPLIT) * b["dX_branch"], "dX")
    for i in range(len(ranks)):
        agree(c["set"].dA[i], b["dA"][i], HALF * b["dA"][i].abs() + (ADD * (N + M + 16) + SPLIT) * b["dA_sum"][i], f"dA[{i}]")


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("shape", CASES)
def test_poisoned_adapter_reaches_its_own_rows_only(gpu_lib, shape, p):
    """Every path, ranks of any kind, dropout: rows that name other adapters, and the other adapters'
    gradients, have the bits that they have beside a finite one."""
    import bit_nf4_quantized_dq_amd as Q

    print(shape, p, flush=True)
    M, N, K, ranks = shape
    c = make(11, M, N, K, ranks, "tokens")
    ids = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    kw = dict(dropout=p, rng=c["rng"] if p else None)
    out = []
    for poison in (False, True):
        if poison:
            A, B = c["A"][1], c["B"][1]
            A[0], A[-1, 7], A[:, -1] = float("nan"), INF, -INF
            B[-1], B[5], B[:, 1] = float("nan"), INF, -INF
        T = torch.empty(M, c["set"].t_width, device="cuda")
        Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], ids, T_save=T, **kw)
        dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], ids, **kw)
        clean = ids != 1
        out.append([Y[clean], T[clean], dX[clean]] + [c["set"].dA[a].clone() for a in (0, 2)] + [c["set"].dB[a].clone() for a in (0, 2)])
    assert all(t.isfinite().all() for t in out[0]) and all(map(torch.equal, *out))
