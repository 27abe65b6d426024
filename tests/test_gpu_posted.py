"""The few-token forwards that hand T from workgroup to workgroup: elements that a workgroup forms for
itself because it stopped waiting.  The number of looks is set from the host: with 0 every workgroup
forms all of its elements while others still post them, so posts come both before and after."""

import pytest
import torch

pytestmark = pytest.mark.gpu
HEAD = 512 * 1024
# d_out, d_in, rows, rank: whole rows to a workgroup
ROWS = [(4096, 2048, 3, 8), (6144, 4096, 2, 64), (4096, 4096, 1, 40), (5120, 4096, 4, 24), (4096, 4096, 4, 16), (4096, 2048, 4, 128),
        (4096, 4096, 1, 16)]
# one token of a large weight: its reduction split or not, a partial row group, ranks of any kind, the longest reduction
STREAM = [(8192, 4096, 1, 16), (8192 + 160, 4096, 1, 40), (14336, 4096, 1, 5), (4096, 14336, 1, 64), (1024, 32768, 1, 24), (57344, 1024, 1, 128)]


@pytest.fixture
def looks(gpu_lib):
    from bit_nf4_quantized_dq_amd._binding import load_library

    put = load_library().qlora_posted_polls
    put.restype = None
    yield put
    put(512)


def make(N, K, M, r, seed=0, codebook="nf4"):
    import bit_nf4_quantized_dq_amd as Q

    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).cuda()  # noqa: E731
    q = Q.quantize(rand(N, K, std=0.02), codebook=codebook)
    return q, rand(M, K).bfloat16(), rand(r, K, std=K**-0.5).bfloat16(), rand(N, r, std=0.1).bfloat16()


def call(c, ws):
    import bit_nf4_quantized_dq_amd as Q

    q, X, A, B = c
    T = torch.empty(X.shape[0], A.shape[0], dtype=torch.bfloat16, device="cuda")
    return Q.linear_fwd(q, X, A, B, 24.0, T_save=T, ws=ws), T


def workspace(c):
    import bit_nf4_quantized_dq_amd as Q

    return Q.new_workspace(Q.workspace_size(Q.OP_FWD, c[1].shape[0], c[0].d_out, c[0].d_in, c[2].shape[0]), "cuda")


def same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


def check_close(c, got):
    import bit_nf4_quantized_dq_amd as Q

    q, X, A, B = c
    T = X.double() @ A.double().T
    Y = X.double() @ Q.dequantize(q).double().T + 24.0 / A.shape[0] * (T @ B.double().T)
    for g, ref in zip(got, (Y, T)):
        assert float((g.double() - ref).norm() / ref.norm()) <= 1e-2


@pytest.mark.parametrize("shape", ROWS + STREAM)
def test_same_bits_whoever_forms_an_element(looks, shape):
    print(shape, flush=True)
    c = make(*shape)
    ws = workspace(c)
    looks(512)
    want = call(c, ws)
    check_close(c, want)
    for n in (0, 0, 1, 2, 0, 512):
        looks(n)
        got = call(c, ws)
        torch.cuda.synchronize()
        assert same(got, want) and not ws[:HEAD].any(), n


@pytest.mark.parametrize("shape", [(4096, 4096, 2, 16), (8192, 4096, 1, 16)])
def test_values_that_are_not_finite(looks, shape):
    c = make(*shape)
    ws = workspace(c)
    c[2][1, 5], c[2][2, 6], c[1][0, 9] = float("nan"), float("inf"), -float("inf")
    want = call(c, ws)
    for n in (0, 1, 512):
        looks(n)
        got = call(c, ws)
        torch.cuda.synchronize()
        assert not ws[:HEAD].any()
        for a, b in zip(got, want):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("shape", [(4096, 4096, 1, 16), (14336, 4096, 1, 40)])
def test_on_streams_at_once_and_replayed(looks, shape):
    cases = [make(*shape, seed=i) for i in range(4)]
    work = [workspace(c) for c in cases]
    want = [call(c, w) for c, w in zip(cases, work)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for n in (512, 0, 1):
        looks(n)
        got = [[] for _ in cases]
        for _ in range(10):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(call(cases[k], work[k]))
        torch.cuda.synchronize()
        for k in range(4):
            assert all(same(g, want[k]) for g in got[k]) and not work[k][:HEAD].any()
    looks(0)
    c, ws = cases[0], work[0]
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            out = [call(c, ws) for _ in range(3)]
    looks(512)
    for turn in range(4):
        c[1].copy_(torch.randn(c[1].shape, generator=torch.Generator().manual_seed(turn)))
        graph.replay()
        torch.cuda.synchronize()
        eager = call(c, ws)
        torch.cuda.synchronize()
        assert all(same(o, eager) for o in out) and not ws[:HEAD].any()


@pytest.mark.parametrize("rank", [16, 40])
def test_linears_of_one_launch(looks, rank):
    """Several weights over the same activations: each linear's row groups take its own columns of T."""
    import bit_nf4_quantized_dq_amd as Q

    shapes = [(8192, 4096), (1024, 4096), (1024, 4096)]
    cases = [make(n, k, 1, rank, seed=i) for i, (n, k) in enumerate(shapes)]
    qs, As, Bs, X = [c[0] for c in cases], [c[2] for c in cases], [c[3] for c in cases], cases[0][1]
    ws = Q.new_workspace(Q.workspace_size_multi(qs, 1, rank), "cuda")

    def run():
        Ts = [torch.empty(1, rank, dtype=torch.bfloat16, device="cuda") for _ in qs]
        return [*Q.linear_fwd_multi(qs, X, As, Bs, 24.0, T_saves=Ts, ws=ws), *Ts]

    want = run()
    for c, y, t in zip(cases, want[:3], want[3:]):
        check_close((c[0], X, c[2], c[3]), (y, t))
    for n in (0, 1, 0, 512):
        looks(n)
        got = run()
        torch.cuda.synchronize()
        assert same(got, want) and not ws[:HEAD].any(), n
