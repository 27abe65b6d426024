"""The frozen linear with many adapters on the GPU against the FP64 oracle: forward, T, backward.

Tolerances.  Each output is an FP32 sum of exact BF16 products, rounded once: half a step of
the output's type on the value (BF16 2^-8, FP32 2^-24), and for the sum at most one 2^-23 (an
addition that truncates) of the sum of absolute terms per addition on a term's way, of which
there are fewer than the reductions' lengths.  FP32 intermediates (T, G) enter products as two
BF16 parts, the second off by half a step of a value that is at most 2^-8 of the whole: 2^-16."""

import pytest
import torch

from oracle import adapters_oracle as AO

pytestmark = pytest.mark.gpu

RNG = (0x1234567890ABCDE, 77)
ADD, HALF, SPLIT = 2.0**-23, 2.0**-8, 2.0**-16


def make(seed, M, N, K, ranks, kind, dq="e4m3", codebook="nf4", grads=True, std=0.02):
    import bit_nf4_quantized_dq_amd as Q

    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).cuda()  # noqa: E731
    q = Q.quantize(rand(N, K, std=std), dq=dq, codebook=codebook)
    A = [rand(r, K, std=K**-0.5).bfloat16() for r in ranks]
    B = [rand(N, r, std=0.1).bfloat16() for r in ranks]
    alpha = [1.0 + 2.0 * i + r for i, r in enumerate(ranks)]
    n = len(ranks)
    if kind == "none":
        ids = None
    elif kind == "tokens":  # each row its own, with some that name none
        ids = torch.randint(-1, n + 1, (M,), generator=gen)
        ids[ids == n] = 1 << 30
    elif kind == "base":
        ids = torch.full((M,), -1)
    else:  # runs of rows; the last adapter has no row
        ids = torch.arange(M) * max(1, n - 1) // M
    ids = None if ids is None else ids.to(torch.int32).cuda()
    more = {}
    if grads:
        # slices of flat buffers, as an optimizer keeps them, and a guard behind the last
        fa = torch.full((sum(ranks) * K + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        fb = torch.full((sum(ranks) * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        more = dict(dA=[t.view(-1, K) for t in fa[:-64].split([r * K for r in ranks])],
                    dB=[t.view(N, -1) for t in fb[:-64].split([r * N for r in ranks])])
    s = Q.AdapterSet(A, B, alpha, **more)
    c = dict(q=q, set=s, A=A, B=B, alpha=alpha, ids=ids, X=rand(M, K).bfloat16(), dY=rand(M, N, std=0.01).bfloat16(),
             rng=torch.tensor(RNG, device="cuda"), what=Q.dequantize(q))
    if grads:
        c["guards"] = [fa[-64:], fb[-64:]]
    return c


def near(got, ref, tol, name):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (name, int(bad.sum()), tuple(bad.nonzero()[0].tolist()), float(got[bad][0]), float(ref[bad][0]),
                           float(tol[bad][0]))


def check_fwd(c, p=0.0, save=True, ws=None):
    import bit_nf4_quantized_dq_amd as Q

    M, K, N = c["X"].shape[0], c["q"].d_in, c["q"].d_out
    # rows behind the last one stay as they were
    Y = torch.full((M + 2, N), 5.0, dtype=torch.bfloat16, device="cuda")
    T = torch.full((M + 2, c["set"].t_width), 5.0, device="cuda") if save else None
    Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=p, rng=c["rng"] if p else None, Y=Y[:M],
                          T_save=None if T is None else T[:M], ws=ws)
    torch.cuda.synchronize()
    ref = AO.fwd(c["what"], c["A"], c["B"], c["alpha"], c["X"], c["ids"], p, RNG)
    r = c["set"].t_width
    near(Y[:M], ref["Y"], HALF * ref["Y"].abs() + ADD * (K + 8) * ref["Y_base"] + (ADD * (K + r + 16) + SPLIT) * ref["Y_branch"], "Y")
    assert (Y[M:] == 5).all()
    if save:
        near(T[:M], ref["T"], 2.0**-23 * ref["T"].abs() + ADD * (K + 8) * ref["T_sum"], "T")
        assert (T[M:] == 5).all()
    return Y[:M], None if T is None else T[:M]


def check_bwd(c, p=0.0, T=None, need_dx=True, ws=None, T_of_oracle=False):
    """T_of_oracle: T is the forward's, and the gradients are those of the oracle's own T."""
    import bit_nf4_quantized_dq_amd as Q

    M, K, N = c["X"].shape[0], c["q"].d_in, c["q"].d_out
    dX = torch.full((M + 2, K), 5.0, dtype=torch.bfloat16, device="cuda")
    got = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"], dropout=p, rng=c["rng"] if p else None, T_saved=T,
                                need_dx=need_dx, dX=dX[:M] if need_dx else None, ws=ws)
    torch.cuda.synchronize()
    ref = AO.bwd(c["what"], c["A"], c["B"], c["alpha"], c["X"], c["dY"], c["ids"], p, RNG,
                 None if T_of_oracle else T)
    r = c["set"].t_width
    assert (got is None) == (not need_dx) and (dX[M:] == 5).all()
    if need_dx:
        near(dX[:M], ref["dX"], HALF * ref["dX"].abs() + ADD * (N + 8) * ref["dX_base"]
             + (ADD * (N + r + 16) + SPLIT) * ref["dX_branch"], "dX")
    else:
        assert (dX == 5).all()
    for i in range(len(c["A"])):
        near(c["set"].dA[i], ref["dA"][i], HALF * ref["dA"][i].abs() + (ADD * (N + M + 16) + SPLIT) * ref["dA_sum"][i], f"dA[{i}]")
        near(c["set"].dB[i], ref["dB"][i], HALF * ref["dB"][i].abs() + (ADD * (K + M + 16) + SPLIT) * ref["dB_sum"][i], f"dB[{i}]")
    for g in c["guards"]:
        assert (g == 7).all()
    return dX[:M]


SHAPES = [  # M, d_out, d_in, ranks, ids
    (1, 16, 64, [8], "none"),
    (1, 4096, 4096, [16] * 4, "tokens"),
    (2, 272, 320, [1, 3], "tokens"),
    (15, 1040, 192, [16, 8, 24], "tokens"),
    (16, 64, 4160, [5, 128, 64], "tokens"),
    (17, 48, 256, [16], "none"),
    (33, 528, 1088, [40, 7], "runs"),
    (64, 256, 512, [16] * 33, "tokens"),
    (65, 80, 64, [100], "tokens"),
    (128, 1024, 704, [12, 9, 1], "runs"),
    (129, 144, 320, [8, 16, 2], "tokens"),
    (200, 512, 2048, [64, 32, 128], "runs"),
    (300, 1040, 576, [17], "none"),
    (257, 272, 1024, [16] * 70, "tokens"),
    (1100, 336, 448, [16, 16, 4], "runs"),
    (777, 2064, 128, [8, 8], "base"),
    (40, 96, 128, [8, 16], "base"),
    # one launch for T and the stream: one and two tiles of 16 ranks
    (1, 48, 4160, [16, 3], "tokens"),
    (1, 272, 192, [32], "none"),
    (1, 4096, 1088, [19, 7], "tokens"),
    (2, 528, 1088, [3, 16], "tokens"),
    (2, 8208, 128, [8], "none"),
    # wide weights: four wavefronts to a workgroup, for each number of row tiles
    (1, 8208, 192, [128, 40], "tokens"),
    (16, 8208, 576, [16, 5], "tokens"),
    (32, 8224, 192, [8] * 20, "tokens"),
    (47, 8208, 320, [16, 24], "tokens"),
    (50, 8208, 192, [7, 16], "tokens"),
    (95, 8208, 128, [16, 8], "runs"),
    (127, 8240, 192, [48, 9, 16], "tokens"),
    (20, 8192, 128, [16, 8], "tokens"),
    (61, 8192, 320, [24, 5], "tokens"),
    (79, 8192, 192, [16, 64], "runs"),
    # up to 128 rows of a large weight
    (65, 8192, 4096, [16], "none"),
    (128, 4112, 8192, [16, 24], "tokens"),
    # several row tiles of a narrow weight
    (96, 112, 1344, [16, 16], "tokens"),
    (113, 64, 4160, [24, 128], "tokens"),
    # products over the codes in tiles of 256 rows, forward and backward, and by the decoded copy
    (520, 6672, 128, [16, 20], "tokens"),
    (513, 128, 6720, [8, 64], "runs"),
    (300, 2064, 192, [16, 24, 7], "tokens"),
    (447, 208, 2112, [9, 40], "runs"),
    (1030, 5776, 64, [16, 20], "tokens"),
    (1030, 64, 5824, [8, 64], "runs"),
    # the gradients' rows in two and four parts
    (2100, 80, 128, [16, 40], "runs"),
    (4111, 48, 64, [128], "none"),
]


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_forward(gpu_lib, i, p):
    print(SHAPES[i], p, flush=True)
    c = make(i, *SHAPES[i], grads=False)
    Y, _ = check_fwd(c, p)
    again, _ = check_fwd(c, p, save=False)
    assert torch.equal(Y, again)


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_backward(gpu_lib, i, p):
    print(SHAPES[i], p, flush=True)
    c = make(100 + i, *SHAPES[i])
    dX = check_bwd(c, p)
    dA, dB = [t.clone() for t in c["set"].dA], [t.clone() for t in c["set"].dB]
    assert torch.equal(dX, check_bwd(c, p))
    assert all(map(torch.equal, dA, c["set"].dA)) and all(map(torch.equal, dB, c["set"].dB))
    # with the forward's T (its sums may be taken in another order than the backward's own)
    _, T = check_fwd(c, p)
    assert torch.equal(dX, check_bwd(c, p, T=T)) and all(map(torch.equal, dA, c["set"].dA))
    check_bwd(c, p, T=T, need_dx=False, T_of_oracle=True)


@pytest.mark.parametrize("dq,codebook", [("none", "nf4"), ("int8", "nf4"), ("e5m2", "fp4"), ("e4m3", "int4"), ("e4m3", "fp4")])
@pytest.mark.parametrize("M", [3, 150])
def test_formats(gpu_lib, M, dq, codebook):
    c = make(M, M, 272, 320, [16, 5], "tokens", dq=dq, codebook=codebook)
    check_fwd(c, 0.1)
    check_bwd(c, 0.1)


@pytest.mark.parametrize("M,N", [(4, 272), (4, 1040), (40, 272), (140, 272)])
def test_values_that_are_not_finite_stay_with_their_rows(gpu_lib, M, N):
    """One adapter holds infinities and NaN: every row that names another, and every other
    adapter's gradient, comes out as if it were finite."""
    import bit_nf4_quantized_dq_amd as Q

    c = make(M, M, N, 320, [16, 8, 24], "tokens")
    ids = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    out = []
    for poison in (False, True):
        if poison:
            c["A"][1][3] = float("nan")
            c["A"][1][:, 7] = float("inf")
            c["B"][1][5] = float("nan")
            c["B"][1][:, 2] = float("-inf")
        Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], ids)
        dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], ids)
        out.append((Y, dX, [c["set"].dA[a].clone() for a in (0, 2)], [c["set"].dB[a].clone() for a in (0, 2)]))
    clean = ids != 1
    (Y0, dX0, dA0, dB0), (Y1, dX1, dA1, dB1) = out
    assert torch.equal(Y0[clean], Y1[clean]) and torch.equal(dX0[clean], dX1[clean])
    assert all(map(torch.equal, dA0, dA1)) and all(map(torch.equal, dB0, dB1))
    assert not torch.isfinite(Y1[~clean].float()).all()


def test_dropped_inputs_that_are_not_finite(gpu_lib):
    """dA takes dropped elements as zeros, whatever they held."""
    import bit_nf4_quantized_dq_amd as Q

    M, K = 70, 320
    c = make(1, M, 272, K, [16, 8], "runs")
    keep = torch.from_numpy(AO.keep_mask(M * K, 0.3, *RNG)).view(M, K).cuda()
    Xn = c["X"].masked_fill(~keep, float("nan"))
    got = []
    for X in (c["X"], Xn):
        T = torch.empty(M, 16, device="cuda")
        Q.linear_adapters_fwd(c["q"], c["set"], X, c["ids"], dropout=0.3, rng=c["rng"], T_save=T)
        Q.linear_adapters_bwd(c["q"], c["set"], X, c["dY"], c["ids"], dropout=0.3, rng=c["rng"])
        got.append([T, *[t.clone() for t in c["set"].dA + c["set"].dB]])
    assert all(map(torch.equal, *got))


def test_one_workspace_for_every_kind_and_shape(gpu_lib):
    """Calls of several shapes and operators on one workspace, and its counters zero after each."""
    import bit_nf4_quantized_dq_amd as Q

    cases = [make(i, *SHAPES[i]) for i in (3, 7, 9, 13, 14, 0)]
    need = max(c["set"].workspace_size(op, c["X"].shape[0]) for c in cases for op in (Q.OP_FWD, Q.OP_BWD))
    ws = Q.new_workspace(need)
    for c in cases + cases[::-1]:
        check_fwd(c, 0.1, ws=ws)
        assert not ws[: 512 * 1024].any()
        check_bwd(c, 0.1, ws=ws)
        assert not ws[: 512 * 1024].any()


def test_agrees_with_the_single_adapter_linear(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    for M in (1, 16, 100, 1100):
        c = make(M, M, 512, 1024, [16], "none")
        Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"])
        one = Q.linear_fwd(c["q"], c["X"], c["A"][0], c["B"][0], c["alpha"][0])
        assert float((Y.float() - one.float()).abs().max() / one.float().abs().max()) <= 1e-2
        dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"])
        dX1, dA1, dB1 = Q.linear_bwd(c["q"], c["X"], c["dY"], c["A"][0], c["B"][0], c["alpha"][0])[:3]
        for a, b in ((dX, dX1), (c["set"].dA[0], dA1), (c["set"].dB[0], dB1)):
            assert float((a.float() - b.float()).abs().max() / b.float().abs().max()) <= 1e-2


@pytest.mark.parametrize("M", [5, 140])
def test_captured_step_draws_new_masks(gpu_lib, M):
    """Forward and backward captured once and replayed: each replay takes the offset that the rng
    tensor and the ids that the ids tensor hold then, and matches the eager call."""
    import bit_nf4_quantized_dq_amd as Q

    c = make(M, M, 272, 320, [16, 24, 8], "tokens")
    T = torch.empty(M, 24, device="cuda")
    Y, dX = torch.empty_like(c["dY"]), torch.empty_like(c["X"])
    ws = Q.new_workspace(max(c["set"].workspace_size(op, M) for op in (Q.OP_FWD, Q.OP_BWD)))

    def step():
        Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=0.2, rng=c["rng"], Y=Y, T_save=T, ws=ws)
        Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"], dropout=0.2, rng=c["rng"], T_saved=T, dX=dX, ws=ws)

    def results():
        return [t.clone() for t in (Y, T, dX, *c["set"].dA, *c["set"].dB)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    seen = []
    for i in range(4):
        c["rng"].copy_(torch.tensor([RNG[0], 100 + i]))
        c["ids"].copy_(torch.randint(-1, 3, (M,), generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = results()
        step()
        torch.cuda.synchronize()
        assert all(map(torch.equal, got, results())), i
        seen.append(got[1])
    assert not torch.equal(seen[0], seen[1])


def test_two_streams_at_once(gpu_lib):
    """Calls on two streams (the binding keeps a workspace for each) give what one stream gives."""
    import bit_nf4_quantized_dq_amd as Q

    cases = [make(i, *SHAPES[i]) for i in (9, 13)]
    want = []
    for c in cases:
        Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"])
        dX = Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"])
        want.append([Y, dX, *[t.clone() for t in c["set"].dA + c["set"].dB]])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(5):
        for k, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                outs[k].append([Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"]),
                                Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"])])
    torch.cuda.synchronize()
    for k, c in enumerate(cases):
        for o in outs[k]:
            assert torch.equal(o[0], want[k][0]) and torch.equal(o[1], want[k][1])
        assert all(map(torch.equal, want[k][2:], c["set"].dA + c["set"].dB))


@pytest.mark.parametrize("shape", [(260, 16, 2**20 + 64, [8, 16], "tokens"), (260, 2**20 + 16, 64, [16, 5], "tokens")])
def test_long_rows(gpu_lib, shape):
    """Rows of more than a million columns, on either side: the gradients look through fewer rows at once."""
    print(shape, flush=True)
    c = make(5, *shape)
    check_fwd(c)
    check_bwd(c)


@pytest.mark.parametrize("i,shape", enumerate([(1, 4096, 4096, [16, 64], "tokens"), (2, 1040, 1088, [16, 8], "tokens"),
                                               (4, 4096, 192, [16, 5, 24], "tokens"), (1, 16384, 128, [30], "none")]))
def test_few_rows_again_and_again(gpu_lib, i, shape):
    """T handed over within a launch: eager calls and replays with other ids, two streams at once, and
    the workspace's head zero after them all."""
    import bit_nf4_quantized_dq_amd as Q

    M = shape[0]
    cases = [make(i, *shape, grads=False), make(i + 10, *shape, grads=False)]
    streams = [torch.cuda.Stream() for _ in cases]
    work = [Q.new_workspace(c["set"].workspace_size(Q.OP_FWD, M)) for c in cases]
    for turn in range(6):
        want = []
        for c in cases:
            if c["ids"] is not None:
                c["ids"].copy_(torch.randint(-1, len(c["A"]), (M,), generator=torch.Generator().manual_seed(turn)))
            Y, T = check_fwd(c, 0.1)
            want.append((Y, T))
        torch.cuda.synchronize()
        got = [[], []]
        for _ in range(10):
            for k, (c, s) in enumerate(zip(cases, streams)):
                with torch.cuda.stream(s):
                    T = torch.empty(M, c["set"].t_width, device="cuda")
                    Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=0.1, rng=c["rng"], T_save=T, ws=work[k])
                    got[k].append((Y, T))
        torch.cuda.synchronize()
        for k in range(2):
            assert not work[k][: 512 * 1024].any()
            for Y, T in got[k]:
                assert torch.equal(Y, want[k][0]) and torch.equal(T, want[k][1])
    c, Y = cases[0], torch.empty(M, shape[1], dtype=torch.bfloat16, device="cuda")
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            for _ in range(5):
                Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=0.1, rng=c["rng"], Y=Y, ws=work[0])
    for turn in range(5):
        if c["ids"] is not None:
            c["ids"].copy_(torch.randint(-1, len(c["A"]), (M,), generator=torch.Generator().manual_seed(50 + turn)))
        c["rng"].copy_(torch.tensor([RNG[0], turn]))
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=0.1, rng=c["rng"])
        assert torch.equal(Y, eager) and not work[0][: 512 * 1024].any()


def test_two_graphs_on_one_workspace(gpu_lib):
    """Two captured calls of different shapes that share a workspace, replayed in turn on one stream."""
    import bit_nf4_quantized_dq_amd as Q

    cases = [make(i, *SHAPES[i]) for i in (13, 6)]
    ws = Q.new_workspace(max(c["set"].workspace_size(op, c["X"].shape[0]) for c in cases for op in (Q.OP_FWD, Q.OP_BWD)))

    def step(c):
        Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], ws=ws)
        return [Y, Q.linear_adapters_bwd(c["q"], c["set"], c["X"], c["dY"], c["ids"], ws=ws), *c["set"].dA, *c["set"].dB]

    want = [[t.clone() for t in step(c)] for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for c in cases:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                outs.append(step(c))
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(map(torch.equal, o, w))


def test_set_of_more_adapters_than_one_launch_describes(gpu_lib):
    """200 adapters (the table is written by three launches); rows name the first, the last and
    those at the seams."""
    import bit_nf4_quantized_dq_amd as Q

    c = make(0, 12, 64, 128, [8] * 200, "tokens")
    c["ids"] = torch.tensor([0, 95, 96, 191, 192, 199, 200, -1, 100, 95, 0, 199], dtype=torch.int32, device="cuda")
    check_fwd(c)
    check_bwd(c)
    assert not c["set"].dA[1].any() and not c["set"].dB[198].any()
    with pytest.raises(ValueError):
        Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"].long())
    with pytest.raises(Q.QLoRAError):
        Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=1.0, rng=c["rng"])
    with pytest.raises(ValueError):
        Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=0.1)
    with pytest.raises(ValueError):
        Q.linear_adapters_bwd(c["q"], Q.AdapterSet(c["A"], c["B"], c["alpha"]), c["X"], c["dY"])
