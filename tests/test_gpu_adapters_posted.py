"""Few rows in one launch: T's elements that a workgroup forms for itself because it stopped waiting for
the workgroup that posts them.  The number of looks is set from the host: with 0 every workgroup
forms all of its elements while others still post them, so posts come both before and after."""

import pytest
import torch

from test_gpu_adapters import RNG, check_fwd, make

pytestmark = pytest.mark.gpu
HEAD = 512 * 1024
# rows, d_out, d_in, ranks, ids: elements on every launch's side of 4 and 8 wavefronts, several ranks, two elements a workgroup
SHAPES = [(1, 4096, 4096, [16] * 4, "tokens"), (1, 4096, 1088, [19, 7], "tokens"), (2, 1040, 1088, [16, 8], "tokens"),
          (2, 8208, 128, [8], "none"), (1, 16384, 128, [30], "none"), (4, 4096, 192, [16, 5, 24], "tokens"),
          (1, 1024, 64, [128, 3], "tokens"), (16, 1024, 320, [8, 8, 8], "tokens"), (1, 48, 4160, [5], "none")]


@pytest.fixture
def looks(gpu_lib):
    from bit_nf4_quantized_dq_amd import _adapters

    put = _adapters._lib().qlora_posted_polls
    put.restype = None
    yield put
    put(512)


def call(c, ws, p):
    import bit_nf4_quantized_dq_amd as Q

    M = c["X"].shape[0]
    T = torch.empty(M, c["set"].t_width, device="cuda")
    Y = Q.linear_adapters_fwd(c["q"], c["set"], c["X"], c["ids"], dropout=p, rng=c["rng"] if p else None, T_save=T, ws=ws)
    return Y, T


def same(a, b):
    return all(torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32)) for x, y in zip(a, b))


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("shape", SHAPES)
def test_same_bits_whoever_forms_an_element(looks, shape, p):
    import bit_nf4_quantized_dq_amd as Q

    print(shape, p, flush=True)
    c = make(3, *shape, grads=False)
    ws = Q.new_workspace(c["set"].workspace_size(Q.OP_FWD, shape[0]))
    looks(512)
    check_fwd(c, p, ws=ws)
    want = call(c, ws, p)
    for n in (0, 0, 1, 2, 0, 512):
        looks(n)
        got = call(c, ws, p)
        torch.cuda.synchronize()
        assert same(got, want) and not ws[:HEAD].any(), n


def test_values_that_are_not_finite(looks):
    """NaN and infinities in T leave the head zero as well."""
    import bit_nf4_quantized_dq_amd as Q

    c = make(4, 2, 4096, 1088, [16, 8], "none", grads=False)
    ws = Q.new_workspace(c["set"].workspace_size(Q.OP_FWD, 2))
    c["A"][0][1, 5] = float("nan")
    c["A"][0][2, 6] = float("inf")
    c["X"][0, 9] = -float("inf")
    want = call(c, ws, 0.0)
    for n in (0, 1, 512):
        looks(n)
        got = call(c, ws, 0.0)
        torch.cuda.synchronize()
        assert not ws[:HEAD].any()
        for a, b in zip(got, want):
            assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


def test_on_streams_at_once_and_replayed(looks):
    """Four launches at once, each on a stream and a workspace of its own, then captured ones."""
    import bit_nf4_quantized_dq_amd as Q

    cases = [make(10 + i, 1, 2896, 1088, [64], "none", grads=False) for i in range(4)]
    work = [Q.new_workspace(c["set"].workspace_size(Q.OP_FWD, 1)) for c in cases]
    want = [call(c, w, 0.2) for c, w in zip(cases, work)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for n in (512, 0, 1):
        looks(n)
        got = [[] for _ in cases]
        for _ in range(10):
            for k, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[k].append(call(cases[k], work[k], 0.2))
        torch.cuda.synchronize()
        for k in range(4):
            assert all(same(g, want[k]) for g in got[k]) and not work[k][:HEAD].any()
    looks(0)
    c, ws = cases[0], work[0]
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            out = [call(c, ws, 0.2) for _ in range(3)]
    looks(512)
    for turn in range(4):
        c["rng"].copy_(torch.tensor([RNG[0], turn]))
        graph.replay()
        torch.cuda.synchronize()
        eager = call(c, ws, 0.2)
        torch.cuda.synchronize()
        assert all(same(o, eager) for o in out) and not ws[:HEAD].any()
