"""Dropout on the GPU against the FP64 oracle.  Each element is one FP32 fused multiply-add by a
scale that is off by at most half an FP32 step, rounded once more to the output's type: half a
step of BF16 (2^-8) or FP32 (2^-24) on the result, and 2^-23 of the product and the sum before."""

import pytest
import torch

from oracle import adapters_oracle as AO

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SEED, OFFSET = 987654321987654321, 5


def rng():
    return torch.tensor([SEED, OFFSET], device="cuda")


def check(out, x, p, residual=None):
    ref = AO.dropout(x, p, (SEED, OFFSET), residual)
    drop = AO.dropout(x, p, (SEED, OFFSET)).abs()
    half = 2.0**-8 if out.dtype == torch.bfloat16 else 2.0**-24
    tol = half * ref.abs() * (1 + 2.0**-20) + 2.0**-23 * (drop + ref.abs())
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 4096, 100003])
@pytest.mark.parametrize("xt,ot,res", [("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                       ("f32", "bf16", False), ("f32", "f32", True), ("f32", "f32", False),
                                       ("f32", "bf16", True), ("bf16", "f32", False)])
def test_against_the_oracle(gpu_lib, n, xt, ot, res):
    import bit_nf4_quantized_dq_amd as Q

    gen = torch.Generator().manual_seed(n)
    # an odd element off the allocation's start, and a guard behind
    buf = torch.full((n + 17,), 3.0, device="cuda", dtype=DT[ot])
    x = torch.randn(n + 1, generator=gen).cuda().to(DT[xt])[1:]
    residual = torch.randn(n + 1, generator=gen).cuda().to(DT[ot])[1:] if res else None
    out = buf[1:n + 1]
    Q.dropout(x, 0.3, rng(), residual=residual, out=out)
    torch.cuda.synchronize()
    check(out, x, 0.3, residual)
    assert (buf[0] == 3) and (buf[n + 1:] == 3).all()
    # where it is written does not change what is dropped
    fresh = Q.dropout(x.clone(), 0.3, rng(), residual=None if residual is None else residual.clone(),
                      out=None if res or xt == ot else torch.empty(n, device="cuda", dtype=DT[ot]))
    assert torch.equal(fresh, out)


@pytest.mark.parametrize("p", [0.0, 1e-7, 2.0**-16, 0.05, 0.5, 0.999, 65535 / 65536])
def test_probabilities(gpu_lib, p):
    import bit_nf4_quantized_dq_amd as Q

    x = torch.randn(3, 5, 333, generator=torch.Generator().manual_seed(1)).cuda()
    check(Q.dropout(x, p, rng()), x, p)


def test_in_place_and_its_gradient(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    x = torch.randn(77, 129, generator=torch.Generator().manual_seed(2)).cuda().bfloat16()
    want = Q.dropout(x, 0.4, rng())
    y = x.clone()
    assert Q.dropout(y, 0.4, rng(), out=y) is y and torch.equal(y, want)
    stream = torch.randn(77, 129, device="cuda")
    want = Q.dropout(x, 0.4, rng(), residual=stream)
    kept = stream.clone()
    assert torch.equal(Q.dropout(x, 0.4, rng(), residual=kept, out=kept), want)
    # the gradient of sum(dout * dropout(x)) by differences: linear, so a step of 1 is exact
    dout = torch.randn(77, 129, device="cuda")
    dx = Q.dropout(dout, 0.4, rng())
    e = torch.zeros(77, 129, device="cuda")
    for at in ((0, 0), (5, 77), (76, 128), (33, 64)):
        e.zero_()[at] = 1.0
        diff = float((dout.double() * Q.dropout(e, 0.4, rng()).double()).sum())
        assert abs(diff - float(dx[at])) <= 2.0**-23 * abs(diff)


def test_dropped_values_that_are_not_finite(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    n = 10001
    keep = torch.from_numpy(AO.keep_mask(n, 0.25, SEED, OFFSET)).cuda()
    for dtype in DT.values():
        x = torch.ones(n, device="cuda", dtype=dtype)
        for bad in (float("nan"), float("inf")):
            got = Q.dropout(x.masked_fill(~keep, bad), 0.25, rng())
            assert torch.equal(got, Q.dropout(x, 0.25, rng())) and not got[~keep].any()


def test_captured_call_takes_the_offset_of_each_replay(gpu_lib):
    import bit_nf4_quantized_dq_amd as Q

    x, out, r = torch.randn(5000, device="cuda"), torch.empty(5000, device="cuda"), rng()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Q.dropout(x, 0.5, r, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            Q.dropout(x, 0.5, r, out=out)
    torch.cuda.synchronize()
    for i in range(4):
        r[1] = i
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, Q.dropout(x, 0.5, r))
        assert torch.equal((got != 0).cpu(), torch.from_numpy(AO.keep_mask(5000, 0.5, SEED, i)))


def test_a_large_tensor(gpu_lib):
    """More blocks than the launch has threads, and the far end of a long tensor."""
    import bit_nf4_quantized_dq_amd as Q

    n = (1 << 25) + 5
    x = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    out = Q.dropout(x, 0.5, rng())
    tail = torch.from_numpy(AO.keep_mask(n, 0.5, SEED, OFFSET)[-4099:]).cuda()
    assert torch.equal(out[-4099:] != 0, tail) and abs(float((out != 0).float().mean()) - 0.5) < 1e-3
