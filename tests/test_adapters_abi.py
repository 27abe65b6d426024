"""CPU-side checks of the adapters' and dropout's entry points: every declared symbol is exported,
sizes and layouts are right, and every argument error returns its status before any launch (no
GPU is touched: the pointers here are never dereferenced)."""

import ctypes
import os
import re

import pytest
import torch

import bit_nf4_quantized_dq_amd as Q
from bit_nf4_quantized_dq_amd import _adapters as AD
from bit_nf4_quantized_dq_amd._binding import _Nf4dq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_adapters.h")
HEAD = 524288
INVALID, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -5
P = ctypes.c_void_p
A, B, C, D, E, W = (P(1 << 20 | i << 12) for i in range(1, 7))  # distinct 16-byte aligned addresses
ODD = P((1 << 20) + 1)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return AD._lib()


def test_every_declared_symbol_is_exported(L):
    names = set(re.findall(r"\bint (qlora_[a-z0-9_]+)\(", open(HEADER).read()))
    assert len(names) == 7
    for n in names:
        assert hasattr(L, n), n


def _set(count=3, d_out=64, d_in=128, max_rank=16, whole=1, grads=1, table=A):
    return AD._AdaptersStruct(table.value if table else None, d_out, d_in, count, max_rank, whole, grads)


def _weight(codes=A, d_out=64, d_in=128, block1=64, codebook=0, dq=0):
    return _Nf4dq(codes.value if codes else None, B.value, C.value, D.value, d_out, d_in, block1, 256, codebook, dq)


def _init(L, count=2, r=(16, 5), alpha=(16.0, 8.0), a=(A, B), b=(C, P((1 << 20) + 2)), da=None, db=None, d_out=64, d_in=128,
          table=W, nbytes=80):
    arr = lambda t, v: None if v is None else (t * len(v))(*[x.value if isinstance(x, P) else x for x in v])  # noqa: E731
    s = AD._AdaptersStruct()
    return L.qlora_adapters_init(count, arr(P, a), arr(P, b), arr(ctypes.c_int32, r), arr(ctypes.c_float, alpha), arr(P, da),
                                 arr(P, db), d_out, d_in, table, nbytes, ctypes.byref(s), None)


@pytest.mark.parametrize("change,status", [
    (dict(count=0), INVALID), (dict(count=4097), INVALID), (dict(r=(16, 0)), INVALID), (dict(r=(129, 5)), INVALID),
    (dict(alpha=(NAN, 8.0)), INVALID), (dict(alpha=(1.0, INF)), INVALID), (dict(a=(A, None)), INVALID),
    (dict(a=(P((1 << 20) + 8), B)), INVALID), (dict(b=(P((1 << 20) + 2), C)), INVALID), (dict(b=(C, ODD)), INVALID),
    (dict(b=(None, C)), INVALID), (dict(da=(A, B)), INVALID), (dict(da=(A, B), db=(A, None)), INVALID),
    (dict(da=(A, ODD), db=(A, B)), INVALID), (dict(d_in=100), SHAPE), (dict(d_out=8), SHAPE), (dict(table=None), WORKSPACE),
    (dict(nbytes=79), WORKSPACE), (dict(table=P((1 << 20) + 8)), INVALID), (dict(a=None), INVALID), (dict(r=None), INVALID),
])
def test_set_refusals(L, change, status):
    assert _init(L, **change) == status


def test_sizes(L):
    n, w = ctypes.c_size_t(), ctypes.c_int64()
    for count in (1, 96, 4096):
        assert L.qlora_adapters_size(count, ctypes.byref(n)) == 0 and n.value == 40 * count
    for rank, width in ((1, 8), (8, 8), (9, 16), (128, 128)):
        assert L.qlora_adapters_t_width(ctypes.byref(_set(max_rank=rank)), ctypes.byref(w)) == 0 and w.value == width
    s = _set(d_out=4096, d_in=4096)
    size = lambda op, M, dq=0: (L.qlora_adapters_workspace_size(op, M, ctypes.byref(s), dq, ctypes.byref(n)), n.value)  # noqa: E731
    assert size(1, 1)[0] == 0 and size(1, 1)[1] < HEAD + (1 << 20)  # few rows: no decoded copy
    assert size(2, 1)[1] < HEAD + (1 << 20)
    for args in ((1, 1, 3), (2, 1, 3), (1, 5000), (2, 5000)):  # many, or a format that only decodes
        assert size(*args)[0] == 0 and size(*args)[1] >= HEAD + 2 * 4096 * 4096
    for args, status in (((0, 1), INVALID), ((3, 1), INVALID), ((1, 0), INVALID), ((1, (1 << 23) + 1), INVALID), ((1, 1, 4), UNSUPPORTED)):
        assert size(*args)[0] == status
    assert L.qlora_adapters_workspace_size(1, 1, None, 0, ctypes.byref(n)) == INVALID
    for bad, status in ((dict(count=0), INVALID), (dict(max_rank=0), INVALID), (dict(max_rank=129), INVALID), (dict(d_in=96), SHAPE)):
        assert L.qlora_adapters_workspace_size(1, 1, ctypes.byref(_set(**bad)), 0, ctypes.byref(n)) == status


def _call(L, bwd, weight=None, aset=None, x=A, dy=B, M=4, ids=C, p=0.0, rng=D, y=E, t=None, ws=W, ws_bytes=1 << 24):
    q, s = weight or _weight(), aset or _set()
    if bwd:
        return L.qlora_adapters_bwd(ctypes.byref(q), ctypes.byref(s), x, dy, M, ids, p, rng, t, y, ws, ws_bytes, None)
    return L.qlora_adapters_fwd(ctypes.byref(q), ctypes.byref(s), x, M, ids, p, rng, y, t, ws, ws_bytes, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(x=P((1 << 20) + 2)), INVALID), (dict(y=P((1 << 20) + 4)), INVALID), (dict(M=0), INVALID),
    (dict(M=(1 << 23) + 1), INVALID), (dict(ids=P((1 << 20) + 2)), INVALID), (dict(p=-0.1), INVALID), (dict(p=1.0), INVALID),
    (dict(p=0.999995), INVALID), (dict(p=NAN), INVALID), (dict(p=0.1, rng=None), INVALID), (dict(p=0.1, rng=P((1 << 20) + 4)), INVALID),
    (dict(t=P((1 << 20) + 4)), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=HEAD), WORKSPACE),
    (dict(ws=P((1 << 20) + 8)), INVALID), (dict(aset=_set(d_in=192)), SHAPE), (dict(aset=_set(table=None)), INVALID),
    (dict(aset=_set(count=5000)), INVALID), (dict(weight=_weight(codes=None)), INVALID), (dict(weight=_weight(block1=32)), UNSUPPORTED),
    (dict(weight=_weight(codebook=5)), UNSUPPORTED), (dict(weight=_weight(d_in=96)), SHAPE),
])
def test_linear_refusals(L, bwd, change, status):
    assert _call(L, bwd, **change) == status


def test_backward_refusals(L):
    assert _call(L, True, dy=None) == INVALID and _call(L, True, aset=_set(grads=0)) == INVALID
    assert _call(L, False, y=None) == INVALID


@pytest.mark.parametrize("off", [0, 16, -16, 1008, -1008])
def test_outputs_over_inputs(L, off):
    """X and dX are 4 x 128, dY and Y 4 x 64 BF16: an output that shares a byte with an input is refused."""
    over = lambda base, span: P(base.value + off) if -span < off < span else None  # noqa: E731
    assert _call(L, True, y=P(A.value + off)) == INVALID  # dX on X (1024 bytes)
    for bwd, change in ((True, dict(y=over(B, 512))), (False, dict(y=over(A, 512)))):
        if change["y"]:
            assert _call(L, bwd, **change) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(n=-1), INVALID), (dict(n=(1 << 40) + 1), INVALID),
    (dict(xt=2), UNSUPPORTED), (dict(ot=-1), UNSUPPORTED), (dict(p=1.0), INVALID), (dict(p=-1.0), INVALID), (dict(rng=None), INVALID),
    (dict(x=ODD), INVALID), (dict(out=P((1 << 20) + 2), ot=1), INVALID), (dict(res=ODD), INVALID),
    (dict(out=P(A.value + 2)), INVALID), (dict(out=A, ot=1), INVALID), (dict(res=P(E.value + 4)), INVALID),
    (dict(out=P(A.value - 198)), INVALID),
])
def test_dropout_refusals(L, change, status):
    a = dict(x=A, xt=0, n=100, p=0.1, rng=D, res=None, out=E, ot=0) | change
    assert L.qlora_dropout(a["x"], a["xt"], a["n"], a["p"], a["rng"], a["res"], a["out"], a["ot"], None) == status


def test_dropout_of_nothing_is_no_call(L):
    assert L.qlora_dropout(None, 0, 0, 0.1, D, None, None, 0, None) == 0


def test_binding_refuses_wrong_tensors_before_the_library():
    bf = torch.bfloat16
    a, b = [torch.zeros(4, 64, dtype=bf)], [torch.zeros(16, 4, dtype=bf)]
    with pytest.raises(ValueError, match="CUDA"):
        Q.AdapterSet(a, b, 8.0)
    for bad in (([], [], 1.0), (a, b * 2, 1.0), (a, b, [1.0, 2.0]), (a, [torch.zeros(16, 5, dtype=bf)], 1.0), (a, [b[0].float()], 1.0)):
        with pytest.raises(ValueError):
            Q.AdapterSet(*bad)
    with pytest.raises(ValueError):
        Q.AdapterSet(a, b, 1.0, dA=a)
    with pytest.raises(ValueError):
        Q.linear_adapters_fwd(None, None, torch.zeros(2, 64, dtype=bf))
    x, rng = torch.zeros(8, dtype=bf), torch.zeros(2, dtype=torch.int64)
    for args, kw in (((x, 0.1, rng), {}), ((x.half(), 0.1, rng), {}), ((x, 0.1, rng[:1]), {}), ((x, 0.1, rng), dict(out=x[:4])),
                     ((x, 0.1, rng), dict(residual=x.double()))):
        with pytest.raises(ValueError):
            Q.dropout(*args, **kw)
