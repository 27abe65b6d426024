"""ctypes binding of include/qlora_adapters.h: the frozen linear with many adapters, the dropout
on their input, and dropout on its own.  Argument marshalling only, as in ``_binding``: torch
tensors provide device memory and the stream, every step runs in the HIP library."""

from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import (DQ_FORMATS, OP_BWD, OP_FWD, QuantizedWeight, _check, _Nf4dq, _ptr, _tokens, _validate,
                       _weight_specs, load_library, quant_sizes)
from ._training import TYPES, _BF16, _F32, _I64, _raw_stream, _right, _workspace


class _AdaptersStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("d_out", ctypes.c_int64), ("d_in", ctypes.c_int64), ("count", ctypes.c_int32),
                ("max_rank", ctypes.c_int32), ("whole", ctypes.c_int32), ("grads", ctypes.c_int32)]


_typed = None


def _lib() -> ctypes.CDLL:
    """The HIP library with the argument types of this header's entry points."""
    global _typed
    if _typed is None:
        L = load_library()
        vp, i64, i32, sz, f, c = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float,
                                  ctypes.c_int)
        P = ctypes.POINTER
        PS, PQ = P(_AdaptersStruct), P(_Nf4dq)
        sig = {
            "qlora_adapters_size": (c, P(sz)),
            "qlora_adapters_init": (c, P(vp), P(vp), P(i32), P(f), P(vp), P(vp), i64, i64, vp, sz, PS, vp),
            "qlora_adapters_t_width": (PS, P(i64)),
            "qlora_adapters_workspace_size": (c, i64, PS, c, P(sz)),
            "qlora_adapters_fwd": (PQ, PS, vp, i64, vp, f, vp, vp, vp, vp, sz, vp),
            "qlora_adapters_bwd": (PQ, PS, vp, vp, i64, vp, f, vp, vp, vp, vp, sz, vp),
            "qlora_dropout": (vp, c, i64, f, vp, vp, vp, c, vp),
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = list(args)
            fn.restype = c
        _typed = L
    return _typed


def _on_device(fn):
    """Calls fn with the device of its first tensor argument current (streams belong to a device)."""

    @functools.wraps(fn)
    def call(*args, **kwargs):
        for t in args:
            if isinstance(t, (torch.Tensor, AdapterSet)):
                index = t.get_device() if isinstance(t, torch.Tensor) else t.device.index
                break
        else:
            index = -1
        if index < 0 or index == torch.cuda.current_device():
            return fn(*args, **kwargs)
        with torch.cuda.device(index):
            return fn(*args, **kwargs)

    return call


def _grads_apart(A, B, dA, dB) -> None:
    """Refuses gradients that share memory with one another or with an adapter (the kernels write
    them in no order)."""
    spans = []
    for name, ts in (("A", A), ("B", B), ("dA", dA or ()), ("dB", dB or ())):
        spans += [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{name}[{i}]") for i, t in enumerate(ts)]
    read, written = (0, ""), (0, "")  # where the spans so far end
    for start, end, name in sorted(spans):
        grad = name[0] == "d"
        for over, other in ((written,) if not grad else (written, read)):
            if start < over:
                raise ValueError(f"{name}: overlaps {other}")
        if grad:
            written = max(written, (end, name))
        else:
            read = max(read, (end, name))


class AdapterSet:
    """The adapters of one linear [d_out, d_in], laid out once: a device table that
    linear_adapters_fwd and _bwd go by.  It holds the tensors (their values may change, their memory
    stays theirs).

    Streams.  The table is written on the stream that is current when the set is made, and its memory
    belongs to that stream, as any tensor's.  Calls on another stream first wait for that one (an
    event, or wait_stream); and the set is kept until such calls have run, and for as long as a
    captured graph that goes by it is replayed.

    A[i] [r_i, d_in], B[i] [d_out, r_i]: contiguous BF16 CUDA tensors, ranks 1..128 that may differ.
    alpha: one number, or one per adapter (the branch is scaled by alpha / r).  dA, dB: tensors of
    the same shapes for the backward's gradients (views of a flat gradient buffer, say), which
    overlap neither each other nor an adapter; None: a set that is not trained."""

    def __init__(self, A, B, alpha, dA=None, dB=None):
        self.A, self.B = list(A), list(B)
        n = len(self.A)
        if n < 1 or len(self.B) != n:
            raise ValueError("AdapterSet: need one A and one B per adapter, at least one")
        if (dA is None) != (dB is None):
            raise ValueError("AdapterSet: need both dA and dB, or neither")
        self.dA, self.dB = (None, None) if dA is None else (list(dA), list(dB))
        if self.dA is not None and (len(self.dA) != n or len(self.dB) != n):
            raise ValueError("AdapterSet: need one dA and one dB per adapter")
        self.alpha = [float(a) for a in alpha] if hasattr(alpha, "__len__") else [float(alpha)] * n
        if len(self.alpha) != n:
            raise ValueError("AdapterSet: need one alpha, or one per adapter")
        for t, name in ((self.A[0], "A[0]"), (self.B[0], "B[0]")):
            if not isinstance(t, torch.Tensor) or t.dim() != 2:
                raise ValueError(f"{name}: need a 2-D tensor")
        self.d_in, self.d_out, self.device = self.A[0].shape[1], self.B[0].shape[0], self.A[0].device
        self.ranks = [t.shape[0] if isinstance(t, torch.Tensor) and t.dim() == 2 else 0 for t in self.A]
        specs = []
        for i, r in enumerate(self.ranks):
            specs += [(self.A[i], _BF16, f"A[{i}]", (r, self.d_in)), (self.B[i], _BF16, f"B[{i}]", (self.d_out, r))]
            if self.dA is not None:
                specs += [(self.dA[i], _BF16, f"dA[{i}]", (r, self.d_in)), (self.dB[i], _BF16, f"dB[{i}]", (self.d_out, r))]
        _validate(specs, self.device)
        _grads_apart(self.A, self.B, self.dA, self.dB)
        L = _lib()
        VP = ctypes.c_void_p * n
        ptrs = lambda ts: None if ts is None else VP(*[t.data_ptr() for t in ts])  # noqa: E731
        size = ctypes.c_size_t()
        _check(L.qlora_adapters_size(n, ctypes.byref(size)), "adapters_size")
        self.table = torch.empty(size.value, dtype=torch.uint8, device=self.device)
        self._struct = _AdaptersStruct()
        self._ref = ctypes.byref(self._struct)
        with torch.cuda.device(self.device):
            _check(L.qlora_adapters_init(n, ptrs(self.A), ptrs(self.B), (ctypes.c_int32 * n)(*self.ranks),
                                         (ctypes.c_float * n)(*self.alpha), ptrs(self.dA), ptrs(self.dB), self.d_out,
                                         self.d_in, self.table.data_ptr(), self.table.numel(), self._ref,
                                         _raw_stream(self.table.get_device())), "adapters_init")
        self.t_width = -(-max(self.ranks) // 8) * 8
        self._sizes: dict = {}

    def __len__(self) -> int:
        return len(self.A)

    def workspace_size(self, op: int, M: int, dq: str = "e4m3") -> int:
        """Workspace bytes of linear_adapters_fwd (OP_FWD) or linear_adapters_bwd (OP_BWD) on M rows."""
        key = (op, M, dq)
        if key not in self._sizes:
            n = ctypes.c_size_t()
            _check(_lib().qlora_adapters_workspace_size(op, M, self._ref, DQ_FORMATS[dq], ctypes.byref(n)),
                   "adapters_workspace_size")
            if len(self._sizes) >= 4096:
                self._sizes.clear()
            self._sizes[key] = n.value
        return self._sizes[key]


def _weight_right(q, index) -> bool:
    """The quantized weight's buffers, contiguous on that GPU, as many elements as its shape and format
    need (what is not so is left to the full check)."""
    nc, n8, n2 = quant_sizes(q.d_out, q.d_in, q.dq)
    c, c8, u8 = q.codes, q.code8, torch.uint8
    try:
        if not (c.dtype is u8 and c.numel() == nc and c.get_device() == index and c.is_contiguous()
                and c8.dtype is u8 and c8.numel() == n8 and c8.get_device() == index and c8.is_contiguous()):
            return False
        s, mu = q.c2s, q.mu
        return q.dq == "none" or (s.dtype is _F32 and 4 * s.numel() == n2 and s.get_device() == index and s.is_contiguous()
                                  and mu.dtype is _F32 and mu.numel() == 1 and mu.get_device() == index)
    except AttributeError:
        return False


def _linear_check(q, adapters, specs, ids, dropout, rng, M):
    if not isinstance(q, QuantizedWeight):
        raise ValueError("weight: need a QuantizedWeight")
    if not isinstance(adapters, AdapterSet):
        raise ValueError("adapters: need an AdapterSet")
    if (adapters.d_out, adapters.d_in) != (q.d_out, q.d_in):
        raise ValueError(f"adapters: of a {adapters.d_out}x{adapters.d_in} linear, the weight is {q.d_out}x{q.d_in}")
    if dropout and rng is None:
        raise ValueError("rng: dropout needs an int64 [2] CUDA tensor (seed, offset)")
    if ids is not None:
        specs.append((ids, torch.int32, "ids", (M,)))
    if rng is not None:
        specs.append((rng, _I64, "rng", (2,)))
    device = adapters.device
    index = device.index
    # what is right passes a short check (a call takes about as long as a small launch)
    if not _weight_right(q, index):
        specs += _weight_specs(q)
    for t, dtype, _, shape in specs:
        if not _right(t, dtype, shape, index):
            _validate(specs, device)


def _struct_of(q):
    return ctypes.byref(q.struct())


def linear_adapters_fwd(q: QuantizedWeight, adapters: AdapterSet, X: torch.Tensor, ids: torch.Tensor | None = None, *,
                        dropout: float = 0.0, rng: torch.Tensor | None = None, Y: torch.Tensor | None = None,
                        T_save: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Y[m] = X[m] w_hat^T + (alpha_a/r_a) T[m] B_a^T, T[m] = drop(X[m]) A_a^T, a = ids[m].

    X [M, d_in] BF16.  ids: int32 [M], the adapter of each row in any order; a number that is none
    (-1, say) leaves its row with the base product; None: adapter 0 for all rows.  dropout: the
    probability to drop an element of the adapters' input, masks from rng: int64 [2] CUDA tensor
    (seed, offset), read when the kernels run.  T_save: FP32 [M, adapters.t_width] that receives T
    for the backward."""
    M = _tokens(X)
    specs = [(X, _BF16, "X", (M, getattr(q, "d_in", 0)))]
    if Y is not None:
        specs.append((Y, _BF16, "Y", (M, getattr(q, "d_out", 0))))
    if T_save is not None:
        specs.append((T_save, _F32, "T_save", (M, getattr(adapters, "t_width", 0))))
    _linear_check(q, adapters, specs, ids, dropout, rng, M)
    return _linear_fwd(X, q, adapters, M, ids, dropout, rng, Y, T_save, ws)


@_on_device
def _linear_fwd(X, q, adapters, M, ids, dropout, rng, Y, T_save, ws):
    index = X.get_device()
    if Y is None:
        Y = torch.empty(M, q.d_out, dtype=_BF16, device=X.device)
    st = _raw_stream(index)
    ws = _workspace(ws, adapters.workspace_size(OP_FWD, M, q.dq), X, index, st)
    status = _lib().qlora_adapters_fwd(_struct_of(q), adapters._ref, X.data_ptr(), M, _ptr(ids), dropout, _ptr(rng),
                                       Y.data_ptr(), _ptr(T_save), ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, "linear_adapters_fwd")
    return Y


def linear_adapters_bwd(q: QuantizedWeight, adapters: AdapterSet, X: torch.Tensor, dY: torch.Tensor,
                        ids: torch.Tensor | None = None, *, dropout: float = 0.0, rng: torch.Tensor | None = None,
                        T_saved: torch.Tensor | None = None, need_dx: bool = True, dX: torch.Tensor | None = None,
                        ws: torch.Tensor | None = None) -> torch.Tensor | None:
    """Backward of linear_adapters_fwd: returns dX (None with need_dx=False) and overwrites the set's
    dA and dB (zeros for adapters that no row names).  ids, dropout and rng as in the forward;
    T_saved: the forward's T_save, None recomputes it."""
    M = _tokens(X)
    specs = [(X, _BF16, "X", (M, getattr(q, "d_in", 0))), (dY, _BF16, "dY", (M, getattr(q, "d_out", 0)))]
    if T_saved is not None:
        specs.append((T_saved, _F32, "T_saved", (M, getattr(adapters, "t_width", 0))))
    if dX is not None:
        if not need_dx:
            raise ValueError("dX: given with need_dx=False")
        specs.append((dX, _BF16, "dX", (M, getattr(q, "d_in", 0))))
    _linear_check(q, adapters, specs, ids, dropout, rng, M)
    if adapters.dA is None:
        raise ValueError("adapters: a set without dA and dB has no backward")
    return _linear_bwd(X, dY, q, adapters, M, ids, dropout, rng, T_saved, need_dx, dX, ws)


@_on_device
def _linear_bwd(X, dY, q, adapters, M, ids, dropout, rng, T_saved, need_dx, dX, ws):
    index = X.get_device()
    if need_dx and dX is None:
        dX = torch.empty_like(X)
    st = _raw_stream(index)
    ws = _workspace(ws, adapters.workspace_size(OP_BWD, M, q.dq), X, index, st)
    status = _lib().qlora_adapters_bwd(_struct_of(q), adapters._ref, X.data_ptr(), dY.data_ptr(), M, _ptr(ids), dropout,
                                       _ptr(rng), _ptr(T_saved), _ptr(dX), ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, "linear_adapters_bwd")
    return dX


@_on_device
def dropout(x: torch.Tensor, p: float, rng: torch.Tensor, *, residual: torch.Tensor | None = None,
            out: torch.Tensor | None = None) -> torch.Tensor:
    """out = residual + drop(x): BF16 or FP32 tensors of one shape; out has the residual's type (x's
    without one, or that of a given out).  Element e (counted row by row) is dropped as rng, an
    int64 [2] CUDA tensor (seed, offset), decides for e alone, so the gradient of x is
    dropout(dout, p, rng) and no mask is kept.  out may be residual, or x of the same type."""
    if not isinstance(x, torch.Tensor) or x.dtype not in TYPES:
        raise ValueError("x: need a bfloat16 or float32 tensor")
    index, shape = x.get_device(), x.shape
    kind = residual.dtype if isinstance(residual, torch.Tensor) else out.dtype if isinstance(out, torch.Tensor) else x.dtype
    if kind not in TYPES:
        raise ValueError(f"{'out' if residual is None else 'residual'}: need a bfloat16 or float32 tensor")
    if not (index >= 0 and x.is_contiguous() and _right(rng, _I64, (2,), index)
            and (residual is None or _right(residual, kind, shape, index)) and (out is None or _right(out, kind, shape, index))):
        specs = [(x, x.dtype, "x", shape), (rng, _I64, "rng", (2,))]
        if residual is not None:
            specs.append((residual, kind, "residual", shape))
        if out is not None:
            specs.append((out, kind, "out", shape))
        _validate(specs, x.device)
    if out is None:
        out = torch.empty_like(x, dtype=kind)
    status = _lib().qlora_dropout(x.data_ptr(), TYPES[x.dtype], x.numel(), p, rng.data_ptr(), _ptr(residual), out.data_ptr(),
                                  TYPES[kind], _raw_stream(index))
    if status:
        _check(status, "dropout")
    return out
