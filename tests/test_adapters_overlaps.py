"""Memory that two arguments of an adapters' call share: refused before any launch where one of them is
written (no GPU is touched: the pointers here are never dereferenced)."""

import ctypes

import pytest
import torch

from bit_nf4_quantized_dq_amd import _adapters as AD
from bit_nf4_quantized_dq_amd._binding import _Nf4dq

INVALID, WORKSPACE = -1, -5
M, N, K, WIDTH = 4, 64, 128, 16
BASE = 1 << 24
SPAN = dict(X=2 * M * K, dY=2 * M * N, Y=2 * M * N, dX=2 * M * K, T=4 * M * WIDTH, ids=4 * M, rng=16)


@pytest.fixture(scope="module")
def L():
    return AD._lib()


def call(L, bwd, over=None):
    """The call on operands 64 KB apart, `over` = {name: address} moved.  Without workspace: a call that
    is not refused for its operands is refused for that."""
    at = {n: BASE + (i << 16) for i, n in enumerate(SPAN)} | (over or {})
    p = {n: ctypes.c_void_p(a) for n, a in at.items()}
    w = ctypes.c_void_p(1 << 20)
    q = _Nf4dq(w.value, w.value, w.value, w.value, N, K, 64, 256, 0, 0)
    s = AD._AdaptersStruct(w.value, N, K, 3, WIDTH, 1, 1)
    if bwd:
        return L.qlora_adapters_bwd(ctypes.byref(q), ctypes.byref(s), p["X"], p["dY"], M, p["ids"], 0.1, p["rng"], p["T"], p["dX"], None, 0, None)
    return L.qlora_adapters_fwd(ctypes.byref(q), ctypes.byref(s), p["X"], M, p["ids"], 0.1, p["rng"], p["Y"], p["T"], None, 0, None)


PAIRS = [(False, out, other) for out in ("Y", "T") for other in ("X", "ids", "rng")] + [(False, "T", "Y")] + \
        [(True, "dX", other) for other in ("X", "dY", "T", "ids", "rng")]


@pytest.mark.parametrize("bwd,out,other", PAIRS)
def test_linears(L, bwd, out, other):
    assert call(L, bwd) == WORKSPACE
    base = BASE + (list(SPAN).index(other) << 16)
    # the output at every 16 bytes around the operand: refused where they share a byte
    for off in range(-SPAN[out] - 32, SPAN[other] + 32, 16):
        want = INVALID if -SPAN[out] < off < SPAN[other] else WORKSPACE
        assert call(L, bwd, {out: base + off}) == want, off


def test_calls_without_the_operand(L):
    q = _Nf4dq(1 << 20, 1 << 20, 1 << 20, 1 << 20, N, K, 64, 256, 0, 0)
    s = AD._AdaptersStruct(1 << 20, N, K, 3, WIDTH, 1, 1)
    at = lambda i: ctypes.c_void_p(BASE + (i << 16))  # noqa: E731
    refs = ctypes.byref(q), ctypes.byref(s)
    assert L.qlora_adapters_fwd(*refs, at(0), M, None, 0.0, None, at(1), None, None, 0, None) == WORKSPACE
    assert L.qlora_adapters_bwd(*refs, at(0), at(1), M, None, 0.0, None, None, None, None, 0, None) == WORKSPACE
    # a generator that is not read may lie anywhere
    assert L.qlora_adapters_fwd(*refs, at(0), M, None, 0.0, at(1), at(1), None, None, 0, None) == WORKSPACE


def test_dropout_over_its_generator(L):
    x, rng = BASE, BASE + (1 << 16)
    for off in (-198, -16, 0, 8, 14):
        assert L.qlora_dropout(x, 0, 100, 0.1, rng, None, rng + off, 0, None) == INVALID, off


def test_gradients_of_a_set():
    flat = torch.zeros(4096, dtype=torch.bfloat16)
    cut = lambda a, n: flat[a:a + n]  # noqa: E731
    A, B, dA, dB = [cut(0, 64), cut(64, 64)], [cut(128, 64), cut(192, 64)], [cut(256, 64), cut(320, 64)], [cut(384, 64), cut(448, 64)]
    AD._grads_apart(A, B, dA, dB)
    AD._grads_apart([A[0], A[0]], [B[0], B[0]], dA, dB)  # one adapter twice, each with gradients of its own
    AD._grads_apart(A, B, None, None)
    for bad in ((A, B, [dA[0], dA[0]], dB), (A, B, dA, [dB[0], cut(447, 64)]), (A, B, dA, [cut(127, 64), dB[1]]), (A, B, A, dB),
                (A, B, [cut(319, 64), cut(319 - 32, 64)], dB), ([cut(256, 512), A[1]], B, dA, dB)):
        with pytest.raises(ValueError, match="overlap"):
            AD._grads_apart(*bad)
