"""CPU-side checks of the training-step entry points: every declared symbol is exported, sizes
and plans are right, and every argument error returns its status before any launch (no GPU is
touched: the pointers here are never dereferenced)."""

import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import bit_nf4_quantized_dq_amd as Q
from bit_nf4_quantized_dq_amd import _training as TR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "qlora_train.h")
HEAD = 524288
INVALID, SHAPE, UNSUPPORTED, WORKSPACE = -1, -2, -3, -5
P = ctypes.c_void_p
A, B, C, D, E, W = (P(1 << 20 | i << 12) for i in range(1, 7))  # distinct 16-byte aligned addresses


@pytest.fixture(scope="module")
def L():
    return TR._lib()


def test_every_declared_symbol_is_exported(L):
    names = set(re.findall(r"\b(qlora_[a-z0-9_]+)\s*\(", open(HEADER).read()))
    own = {n for n in names if n.startswith(("qlora_norm_residual", "qlora_logps", "qlora_token", "qlora_pref", "qlora_grad",
                                             "qlora_adamw_step_clipped"))}
    assert len(own) == 13
    for n in own:
        assert hasattr(L, n), n


def _fwd(L, x=A, y=B, M=4, d=64, type=0, post=1, w_post=C, gate=D, rows=4, w_pre=C, scale=1.0, eps=1e-5, xo=E, h=W):
    return L.qlora_norm_residual_fwd(x, y, M, d, type, post, w_post, gate, rows, w_pre, scale, eps, xo, h, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(M=0), INVALID), (dict(M=1 << 24), INVALID), (dict(d=0), SHAPE), (dict(d=8193), SHAPE),
    (dict(type=2), UNSUPPORTED), (dict(type=-1), UNSUPPORTED), (dict(xo=None, h=None, w_pre=None), INVALID),
    (dict(h=None), INVALID), (dict(y=None), INVALID), (dict(y=None, post=0, w_post=None), INVALID), (dict(post=0), INVALID),
    (dict(rows=0), INVALID), (dict(rows=-3), INVALID), (dict(scale=float("inf")), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=P((1 << 20) + 1)), INVALID), (dict(x=P((1 << 20) + 2), type=1), INVALID),
    (dict(h=P((1 << 20) + 1)), INVALID), (dict(gate=P((1 << 20) + 1)), INVALID),
])
def test_norm_forward_refusals(L, change, status):
    assert _fwd(L, **change) == status


def _bwd(L, x=A, y=B, dh=C, dxo=D, M=4, d=64, type=0, post=1, w_post=C, gate=D, rows=4, w_pre=C, scale=1.0, eps=1e-5,
         dx=E, dy=W, dwp=A, dg=B, dw=C, ws=A, ws_bytes=1 << 22):
    return L.qlora_norm_residual_bwd(x, y, dh, dxo, M, d, type, post, w_post, gate, rows, w_pre, scale, eps, dx, dy, dwp,
                                     dg, dw, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(dh=None, dxo=None), INVALID), (dict(x=None), INVALID), (dict(dh=None), INVALID),
    (dict(dh=None, w_pre=None), INVALID), (dict(dx=None, dy=None, dwp=None, dg=None, dw=None), INVALID),
    (dict(y=None, post=0, w_post=None, gate=None), INVALID), (dict(post=0, w_post=None), INVALID),
    (dict(gate=None), INVALID), (dict(d=9000), SHAPE), (dict(type=7), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=HEAD), WORKSPACE), (dict(ws=P((1 << 20) + 8)), INVALID), (dict(dx=P(4097)), INVALID),
])
def test_norm_backward_refusals(L, change, status):
    assert _bwd(L, **change) == status


def _pref(L, x=A, lab=B, ref=C, pairs=2, S=8, V=100, type=0, beta=0.1, eps=0.0, scale=1.0, loss=C, ratios=D, lps=E, dx=None,
          ws=A, ws_bytes=1 << 22):
    return L.qlora_preference_loss(x, lab, ref, pairs, S, V, type, beta, eps, scale, loss, ratios, lps, dx, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(lab=None), INVALID), (dict(lab=P(4100)), INVALID), (dict(pairs=0), INVALID),
    (dict(S=0), INVALID), (dict(pairs=1 << 22), INVALID), (dict(pairs=1 << 12, S=1 << 12), INVALID), (dict(V=0), SHAPE),
    (dict(V=(1 << 22) + 1), SHAPE), (dict(type=3), UNSUPPORTED), (dict(beta=float("nan")), INVALID),
    (dict(eps=-0.1), INVALID), (dict(eps=1.5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(loss=None), INVALID), (dict(ratios=None), INVALID), (dict(lps=None), INVALID),
    (dict(ref=P(4098)), INVALID), (dict(dx=P((1 << 20 | 1 << 12) + 2)), INVALID), (dict(dx=P((1 << 20 | 1 << 12) - 64)), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=HEAD), WORKSPACE),
])
def test_preference_refusals(L, change, status):
    assert _pref(L, **change) == status


def test_token_logps_refusals(L):
    f = lambda x=A, lab=B, rows=4, V=10, type=0, out=C, ws=A, n=1 << 22: L.qlora_token_logps(x, lab, rows, V, type, out, ws, n, None)  # noqa: E731
    assert f(out=None) == f(x=None) == f(rows=0) == f(rows=1 << 24) == f(out=P(4097)) == INVALID
    assert f(V=0) == SHAPE and f(type=9) == UNSUPPORTED and f(ws=None) == f(n=HEAD) == WORKSPACE


def _list(L, sizes, types=None, ptrs=None, out=None, out_types=None, table=A, table_bytes=1 << 20):
    n = len(sizes)
    arr = lambda ct, v: None if v is None else (ct * n)(*v)  # noqa: E731
    s = TR._GradListStruct()
    st = L.qlora_gradlist_init(n, arr(P, ptrs or [1 << 20] * n), arr(ctypes.c_int32, types or [0] * n),
                               arr(ctypes.c_int64, sizes), arr(P, out), arr(ctypes.c_int32, out_types), table, table_bytes,
                               ctypes.byref(s), None)
    return st


def test_grad_list_refusals(L):
    n = ctypes.c_size_t()
    size = lambda v: L.qlora_gradlist_size(len(v), (ctypes.c_int64 * len(v))(*v), ctypes.byref(n))  # noqa: E731
    assert size([0, 1, 16384, 16385]) == 0 and n.value == 24 * 4
    assert size([]) == 0 and n.value == 0
    assert size([-1]) == INVALID and size([1 << 50]) == SHAPE and size([1 << 37] * 3) == SHAPE
    assert L.qlora_gradlist_size(-1, None, ctypes.byref(n)) == INVALID
    assert L.qlora_gradlist_size(1, None, ctypes.byref(n)) == INVALID
    assert _list(L, [4], types=[5]) == UNSUPPORTED
    assert _list(L, [4], ptrs=[4097]) == INVALID and _list(L, [4], types=[1], ptrs=[4098]) == INVALID
    assert _list(L, [4], ptrs=[1 << 20], out=[1 << 20], out_types=[1]) == INVALID  # in place, another type
    assert _list(L, [4], out=[None], out_types=[0]) == INVALID
    assert _list(L, [40000], table_bytes=24) == WORKSPACE and _list(L, [4], table=None) == WORKSPACE
    assert _list(L, [4], table=P(4100)) == INVALID
    s = TR._GradListStruct(None, 3)
    assert L.qlora_grad_norm(ctypes.byref(s), A, B, 1 << 22, None) == INVALID
    s = TR._GradListStruct(1 << 20, 3)
    assert L.qlora_grad_norm(None, A, B, 1 << 22, None) == INVALID
    assert L.qlora_grad_norm(ctypes.byref(s), None, B, 1 << 22, None) == INVALID
    assert L.qlora_grad_norm(ctypes.byref(s), A, B, HEAD, None) == WORKSPACE
    for bad in (-1.0, float("inf"), float("nan")):
        assert L.qlora_grad_clip(ctypes.byref(s), bad, A, B, 1 << 22, None) == INVALID


def test_clipped_adamw_refusals(L):
    f = lambda master=A, n=4, step=1, lr=1e-3, norm=E, mx=1.0, grad=D: L.qlora_adamw_step_clipped(  # noqa: E731
        master, B, C, grad, None, n, step, lr, 0.9, 0.999, 1e-8, 0.0, norm, mx, None)
    assert f(n=-1) == f(step=0) == f(lr=-1.0) == f(master=None) == f(norm=None) == f(mx=-1.0) == INVALID
    assert f(mx=float("inf")) == f(mx=float("nan")) == f(grad=P(4100)) == INVALID
    assert f(n=0) == 0


def test_workspace_sizes():
    """The counter head and the parts after it."""
    # 4096 rows of 8192: 256 segments of 16 rows, three FP32 partials each
    assert Q.norm_residual_workspace_size(4096, 8192, 4096) == HEAD + 3 * 256 * 8192 * 4
    assert Q.norm_residual_workspace_size(1, 64) == HEAD + 3 * 64 * 4
    assert Q.logps_workspace_size(4096, 32768) == HEAD + 8 * 4096           # whole rows
    assert Q.logps_workspace_size(16, 131072) == HEAD + 8 * 16 * 16 + 256   # sixteen parts, label logits
    assert Q.preference_workspace_size(4, 512, 32768) == HEAD + (8 + 8) * 4096 + 256
    for bad in ((0, 64, 0), (1 << 24, 64, 0)):
        with pytest.raises(Q.QLoRAError) as e:
            Q.norm_residual_workspace_size(*bad)
        assert e.value.status == INVALID
    with pytest.raises(Q.QLoRAError) as e:
        Q.preference_workspace_size(4, 512, 1 << 23)
    assert e.value.status == SHAPE


def test_python_refusals():
    """Types, shapes and placement are refused before a pointer crosses."""
    bf = torch.bfloat16
    x, y, w = torch.zeros(4, 8, dtype=bf), torch.zeros(4, 8, dtype=bf), torch.zeros(8, dtype=bf)
    bad = [
        lambda: Q.norm_residual_fwd(x, y),                                           # on the CPU
        lambda: Q.norm_residual_fwd(x.half(), y), lambda: Q.norm_residual_fwd(x[0], y),
        lambda: Q.norm_residual_fwd(x, y.float()), lambda: Q.norm_residual_fwd(x, y[:2]),
        lambda: Q.norm_residual_fwd(x.t().contiguous().t(), y), lambda: Q.norm_residual_fwd(x, y, gate=w[None]),
        lambda: Q.norm_residual_fwd(x, y, gate=w[None], gate_rows=2), lambda: Q.norm_residual_fwd(x, y, w_pre=w[:4]),
        lambda: Q.norm_residual_fwd(x, y, pre_norm=False, h=y), lambda: Q.norm_residual_bwd(None, y, x, None),
        lambda: Q.norm_residual_bwd(x, y, x.float(), x), lambda: Q.norm_residual_bwd(x, y, x, x.float()),
        lambda: Q.token_logps(x, torch.zeros(4)), lambda: Q.token_logps(x, torch.zeros(3, dtype=torch.int64)),
        lambda: Q.token_logps(x.double(), torch.zeros(4, dtype=torch.int64)),
        lambda: Q.preference_loss(x, torch.zeros(4, dtype=torch.int64), None, 0.1),
        lambda: Q.preference_loss(torch.zeros(3, 2, 5), torch.zeros(3, 2, dtype=torch.int64), None, 0.1),
        lambda: Q.preference_loss(torch.zeros(2, 2, 5), torch.zeros(2, 2, dtype=torch.int64), torch.zeros(2, 1), 0.1),
        lambda: Q.preference_loss(torch.zeros(2, 2, 5), torch.zeros(2, 2, dtype=torch.int64), None, 0.1, need_grad=False,
                                  dlogits=torch.zeros(2, 2, 5)),
        lambda: Q.GradList([]), lambda: Q.GradList([x]), lambda: Q.GradList([x.half()]), lambda: Q.GradList([None]),
        lambda: Q.GradList([x], out=[]), lambda: Q.grad_norm([x]), lambda: Q.grad_clip(x, 1.0),
        lambda: Q.adamw_step_clipped(x.float(), x.float(), x.float(), x, torch.zeros(1), 1.0, 1, 1e-3),
        lambda: Q.adamw_step_clipped(None, None, None, None, None, 1.0, 1, 1e-3),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)


def test_package_imports_on_a_torch_without_gpu_support():
    """A CPU build of torch has no stream functions: the package still imports (its generators and
    codebooks need no GPU), and the operators refuse as they do for any CPU tensor."""
    code = ("import torch\n"
            "del torch._C._cuda_getCurrentRawStream\n"
            "import bit_nf4_quantized_dq_amd as Q\n"
            "x = torch.zeros(4, 8)\n"
            "try:\n    Q.norm_residual_fwd(x)\nexcept ValueError:\n    print('refused')\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "refused", out.stderr


def test_alignment_of_each_operand(L):
    """What the header promises: elements' alignment passes (the call goes on to its next check),
    the optimizer's buffers need a vector's."""
    odd16, odd32 = P((1 << 20) + 2), P((1 << 20) + 4)
    assert _bwd(L, x=odd32, dxo=odd32, dx=odd32, y=odd16, dh=odd16, w_post=odd16, gate=odd16, w_pre=odd16, dy=odd16,
                dwp=odd16, dg=odd16, dw=odd16, type=1, ws=None) == WORKSPACE
    assert _pref(L, x=odd16, dx=odd16, ref=odd32, loss=odd32, ratios=odd32, lps=odd32, ws=None) == WORKSPACE
    assert _list(L, [4], ptrs=[(1 << 20) + 2], table=None) == WORKSPACE
    step = lambda master=A, m=B, v=C, grad=D, param=E, norm=None: L.qlora_adamw_step_clipped(  # noqa: E731
        master, m, v, grad, param, 4, 1, 1e-3, 0.9, 0.999, 1e-8, 0.0, norm, 1.0, None)
    for name in ("master", "m", "v"):
        assert step(**{name: P((1 << 20) + 8)}, norm=W) == INVALID
    for name in ("grad", "param"):
        assert step(**{name: P((1 << 20) + 4)}, norm=W) == INVALID
