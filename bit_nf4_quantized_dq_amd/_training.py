"""ctypes binding of include/qlora_train.h: block norms, the preference loss and gradient
clipping.  Argument marshalling only, as in ``_binding``: torch tensors provide device memory
and the stream, every step runs in the HIP library."""

from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _check, _check_ws, _ptr, _validate, _WS, load_library

TYPES = {torch.bfloat16: 0, torch.float32: 1}


class _GradListStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("chunks", ctypes.c_int64)]


_typed = None


def _lib() -> ctypes.CDLL:
    """The HIP library with the argument types of this header's entry points."""
    global _typed
    if _typed is None:
        L = load_library()
        vp, i64, i32, sz, f, c = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float,
                                  ctypes.c_int)
        P = ctypes.POINTER
        PL = P(_GradListStruct)
        sig = {
            "qlora_norm_residual_fwd": (vp, vp, i64, i64, c, c, vp, vp, i64, vp, f, f, vp, vp, vp),
            "qlora_norm_residual_workspace_size": (i64, i64, i64, P(sz)),
            "qlora_norm_residual_bwd": (vp, vp, vp, vp, i64, i64, c, c, vp, vp, i64, vp, f, f, vp, vp, vp, vp, vp, vp,
                                        sz, vp),
            "qlora_logps_workspace_size": (i64, i64, P(sz)),
            "qlora_token_logps": (vp, vp, i64, i64, c, vp, vp, sz, vp),
            "qlora_preference_workspace_size": (i64, i64, i64, P(sz)),
            "qlora_preference_loss": (vp, vp, vp, i64, i64, i64, c, f, f, f, vp, vp, vp, vp, vp, sz, vp),
            "qlora_gradlist_size": (c, P(i64), P(sz)),
            "qlora_gradlist_init": (c, P(vp), P(i32), P(i64), P(vp), P(i32), vp, sz, PL, vp),
            "qlora_grad_workspace_size": (PL, P(sz)),
            "qlora_grad_norm": (PL, vp, vp, sz, vp),
            "qlora_grad_clip": (PL, f, vp, vp, sz, vp),
            "qlora_adamw_step_clipped": (vp, vp, vp, vp, vp, i64, i64, f, f, f, f, f, vp, f, vp),
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = list(args)
            fn.restype = ctypes.c_int
        _typed = L
    return _typed


# The small calls here take a few microseconds on the device, about as long as their checks, so
# the marshalling below avoids what costs one on the host: the stream's handle is asked for
# directly (0.1 us; through a Stream object 2 us), and what is right passes a short check.
# (A CPU build of torch lacks it; every call has refused its tensors by then.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_BF16, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64


def _right(t, dtype, shape, index) -> bool:
    """A contiguous tensor of that dtype and shape on that GPU (one on the CPU has the number -1)."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous())


def _tensors(specs, device) -> None:
    """_validate, with a quick pass first."""
    if device is not None and device.type == "cuda":
        index = device.index
        for t, dtype, _, shape in specs:
            if not _right(t, dtype, shape, index):
                break
        else:
            return
    _validate(specs, device)


def _workspace(ws, nbytes: int, t: torch.Tensor, index: int, stream: int) -> torch.Tensor:
    """The caller's workspace, checked, or the binding's own for this device and stream."""
    if ws is not None:
        _check_ws(ws, t.device)
        return ws
    buf = _WS._bufs.get((index, stream, "train"))
    return buf if buf is not None and buf.numel() >= nbytes else _WS.get(nbytes, t.device, "train")


def _type(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in TYPES:
        raise ValueError(f"{name}: need a bfloat16 or float32 tensor")
    return TYPES[t.dtype]


def _size(fn: str, *args) -> int:
    n = ctypes.c_size_t()
    _check(getattr(_lib(), fn)(*args, ctypes.byref(n)), fn[len("qlora_"):])
    return n.value


@functools.lru_cache(maxsize=4096)
def norm_residual_workspace_size(M: int, d: int, gate_rows: int = 0) -> int:
    return _size("qlora_norm_residual_workspace_size", M, d, gate_rows)


@functools.lru_cache(maxsize=4096)
def logps_workspace_size(rows: int, V: int) -> int:
    return _size("qlora_logps_workspace_size", rows, V)


@functools.lru_cache(maxsize=4096)
def preference_workspace_size(pairs: int, S: int, V: int) -> int:
    return _size("qlora_preference_workspace_size", pairs, S, V)


def _norm_specs(x, y, w_post, gate, gate_rows, w_pre, M, d, x_name):
    bf16 = torch.bfloat16
    specs = []
    if x is not None:
        specs.append((x, x.dtype, x_name, (M, d)))
    if y is not None:
        specs.append((y, bf16, "y", (M, d)))
    if w_post is not None:
        specs.append((w_post, bf16, "w_post", (d,)))
    if w_pre is not None:
        specs.append((w_pre, bf16, "w_pre", (d,)))
    if gate is not None:
        if int(gate_rows) < 1:
            raise ValueError("gate_rows: need the number of rows that share a gate row")
        specs.append((gate, bf16, "gate", (-(-M // int(gate_rows)), d)))
    return specs


def norm_residual_fwd(x: torch.Tensor, y: torch.Tensor | None = None, *, post_norm: bool = False,
                      w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None, gate_rows: int = 0,
                      pre_norm: bool = True, w_pre: torch.Tensor | None = None, res_scale: float = 1.0,
                      eps: float = 1e-5, x_out: torch.Tensor | None = None, h: torch.Tensor | None = None):
    """The boundary between two blocks: x' = res_scale x + gate * (norm of) y, h = norm of x'.

    x [M, d] BF16 or FP32 (the residual stream), y [M, d] BF16 (the block's output) or None.
    post_norm: norm y first (w_post [d] BF16, or ones).  gate [ceil(M / gate_rows), d] BF16: one
    row for each gate_rows rows of the stream.  pre_norm: also give the next block's input h
    (w_pre [d] BF16, or ones).  x_out may be x.  Returns (x_out, h), h None without pre_norm."""
    kind = _type(x, "x")
    if x.dim() != 2:
        raise ValueError("x: need a 2-D [M, d] tensor")
    shape = M, d = x.shape
    index = x.get_device()
    if not (index >= 0 and x.is_contiguous() and (y is None or _right(y, _BF16, shape, index))
            and (w_post is None or _right(w_post, _BF16, (d,), index)) and (w_pre is None or _right(w_pre, _BF16, (d,), index))
            and (gate is None or (gate_rows >= 1 and _right(gate, _BF16, (-(-M // gate_rows), d), index)))
            and (x_out is None or _right(x_out, x.dtype, shape, index))
            and (h is None or (pre_norm and _right(h, _BF16, shape, index)))):
        specs = _norm_specs(x, y, w_post, gate, gate_rows, w_pre, M, d, "x")
        if x_out is not None:
            specs.append((x_out, x.dtype, "x_out", (M, d)))
        if h is not None:
            if not pre_norm:
                raise ValueError("h: given without pre_norm")
            specs.append((h, _BF16, "h", (M, d)))
        _validate(specs, x.device)
    if x_out is None:
        x_out = torch.empty_like(x)
    if pre_norm and h is None:
        h = torch.empty_like(x, dtype=_BF16) if y is None else torch.empty_like(y)
    status = _lib().qlora_norm_residual_fwd(
        x.data_ptr(), None if y is None else y.data_ptr(), M, d, kind, post_norm,
        None if w_post is None else w_post.data_ptr(), None if gate is None else gate.data_ptr(), gate_rows,
        None if w_pre is None else w_pre.data_ptr(), res_scale, eps, x_out.data_ptr(),
        None if h is None else h.data_ptr(), _raw_stream(index))
    if status:
        _check(status, "norm_residual_fwd")
    return x_out, h


def norm_residual_bwd(x_out: torch.Tensor | None, y: torch.Tensor | None, dh: torch.Tensor | None,
                      dx_out: torch.Tensor | None = None, *, post_norm: bool = False,
                      w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None, gate_rows: int = 0,
                      w_pre: torch.Tensor | None = None, res_scale: float = 1.0, eps: float = 1e-5,
                      need_weights: bool = True, need_gate: bool = True, dx: torch.Tensor | None = None,
                      dy: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Backward of norm_residual_fwd: returns (dx, dy, dw_post, dgate, dw_pre).

    x_out is the forward's x', dh the gradient of h (None: h was not used) and dx_out the
    gradient that reaches x' from later blocks (None: none).  dx may be dx_out.  dy is None
    without y, dw_post and dw_pre without their weight (or with need_weights=False), dgate
    without a gate (or with need_gate=False)."""
    stream = x_out if x_out is not None else dx_out
    kind = _type(stream, "x_out")
    if stream.dim() != 2:
        raise ValueError("x_out: need a 2-D [M, d] tensor")
    shape = M, d = stream.shape
    index, dtype = stream.get_device(), stream.dtype
    if not (index >= 0 and stream.is_contiguous() and (y is None or _right(y, _BF16, shape, index))
            and (dh is None or _right(dh, _BF16, shape, index)) and (dx_out is None or _right(dx_out, dtype, shape, index))
            and (w_post is None or _right(w_post, _BF16, (d,), index)) and (w_pre is None or _right(w_pre, _BF16, (d,), index))
            and (gate is None or (gate_rows >= 1 and _right(gate, _BF16, (-(-M // gate_rows), d), index)))
            and (dx is None or _right(dx, dtype, shape, index)) and (dy is None or _right(dy, _BF16, shape, index))):
        specs = _norm_specs(x_out, y, w_post, gate, gate_rows, w_pre, M, d, "x_out")
        for t, kind_of, name in ((dh, _BF16, "dh"), (dx_out, dtype, "dx_out"), (dx, dtype, "dx"), (dy, _BF16, "dy")):
            if t is not None:
                specs.append((t, kind_of, name, (M, d)))
        _validate(specs, stream.device)
    if dx is None:
        dx = torch.empty_like(stream)
    if y is not None and dy is None:
        dy = torch.empty_like(y)
    dw_post = torch.empty_like(w_post) if w_post is not None and need_weights else None
    dw_pre = torch.empty_like(w_pre) if w_pre is not None and need_weights else None
    dgate = torch.empty_like(gate) if gate is not None and need_gate else None
    rows = gate_rows if gate is not None else 0
    st = _raw_stream(index)
    ws = _workspace(ws, norm_residual_workspace_size(M, d, rows), stream, index, st)
    status = _lib().qlora_norm_residual_bwd(
        None if x_out is None else x_out.data_ptr(), None if y is None else y.data_ptr(),
        None if dh is None else dh.data_ptr(), None if dx_out is None else dx_out.data_ptr(), M, d, kind, post_norm,
        None if w_post is None else w_post.data_ptr(), None if gate is None else gate.data_ptr(), rows,
        None if w_pre is None else w_pre.data_ptr(), res_scale, eps, dx.data_ptr(), None if dy is None else dy.data_ptr(),
        None if dw_post is None else dw_post.data_ptr(), None if dgate is None else dgate.data_ptr(),
        None if dw_pre is None else dw_pre.data_ptr(), ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, "norm_residual_bwd")
    return dx, dy, dw_post, dgate, dw_pre


def token_logps(logits: torch.Tensor, labels: torch.Tensor, logps: torch.Tensor | None = None,
                ws: torch.Tensor | None = None) -> torch.Tensor:
    """FP32 log-probability of each row's label: logits [..., V] BF16 or FP32, labels [...] int64.
    A label outside [0, V) (-100, say) leaves its row out: 0, and its logits are not read."""
    kind = _type(logits, "logits")
    if logits.dim() < 1:
        raise ValueError("logits: need [..., V]")
    lead, V, dev = logits.shape[:-1], logits.shape[-1], logits.device
    specs = [(logits, logits.dtype, "logits", logits.shape), (labels, torch.int64, "labels", lead)]
    if logps is not None:
        specs.append((logps, torch.float32, "logps", lead))
    _tensors(specs, dev)
    rows = labels.numel()
    if logps is None:
        logps = torch.empty_like(labels, dtype=_F32)
    index = logits.get_device()
    st = _raw_stream(index)
    ws = _workspace(ws, logps_workspace_size(rows, V), logits, index, st)
    status = _lib().qlora_token_logps(logits.data_ptr(), labels.data_ptr(), rows, V, kind, logps.data_ptr(),
                                      ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, "token_logps")
    return logps


def preference_loss(logits: torch.Tensor, labels: torch.Tensor, ref_logps: torch.Tensor | None, beta: float,
                    label_smoothing: float = 0.0, grad_scale: float = 1.0, need_grad: bool = True,
                    dlogits: torch.Tensor | None = None, ws: torch.Tensor | None = None):
    """Preference loss of answer pairs: returns (loss [1], log_ratios [2P], logps [2P, S], dlogits).

    logits [2P, S, V] BF16 or FP32 (the P chosen answers, then their rejected ones), labels
    [2P, S] int64 (already shifted; outside [0, V): left out), ref_logps [2P, S] FP32 from
    token_logps on the reference model, or None for zeros.  dlogits may be logits (overwritten);
    it is None with need_grad=False.  The gradient is that of grad_scale * loss."""
    kind = _type(logits, "logits")
    if logits.dim() != 3 or logits.shape[0] % 2 or logits.shape[0] == 0:
        raise ValueError("logits: need [2 pairs, S, V]")
    n, S, V = logits.shape
    dev = logits.device
    index = logits.get_device()
    if not (index >= 0 and logits.is_contiguous() and _right(labels, _I64, (n, S), index)
            and (ref_logps is None or _right(ref_logps, _F32, (n, S), index))
            and (dlogits is None or (need_grad and _right(dlogits, logits.dtype, logits.shape, index)))):
        specs = [(logits, logits.dtype, "logits", (n, S, V)), (labels, _I64, "labels", (n, S))]
        if ref_logps is not None:
            specs.append((ref_logps, _F32, "ref_logps", (n, S)))
        if dlogits is not None:
            if not need_grad:
                raise ValueError("dlogits: given with need_grad=False")
            specs.append((dlogits, logits.dtype, "dlogits", (n, S, V)))
        _validate(specs, dev)
    loss = torch.empty(1, dtype=_F32, device=dev)
    log_ratios = torch.empty(n, dtype=_F32, device=dev)
    logps = torch.empty_like(labels, dtype=_F32)
    if need_grad and dlogits is None:
        dlogits = torch.empty_like(logits)
    st = _raw_stream(index)
    ws = _workspace(ws, preference_workspace_size(n // 2, S, V), logits, index, st)
    status = _lib().qlora_preference_loss(
        logits.data_ptr(), labels.data_ptr(), None if ref_logps is None else ref_logps.data_ptr(), n // 2, S, V, kind, beta,
        label_smoothing, grad_scale, loss.data_ptr(), log_ratios.data_ptr(), logps.data_ptr(),
        None if dlogits is None else dlogits.data_ptr(), ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, "preference_loss")
    return loss, log_ratios, logps, dlogits


class GradList:
    """A model's gradient tensors, laid out once: a device table that grad_norm and grad_clip go
    by.  It holds the tensors (their values may change, their memory stays theirs); the table
    is written on the stream that is current when the list is made.

    tensors: contiguous BF16 or FP32 CUDA tensors.  out: where grad_clip writes, one tensor of
    the same size for each (BF16 or FP32); None clips in place."""

    def __init__(self, tensors, out=None):
        self.tensors = list(tensors)
        self.out = None if out is None else list(out)
        if self.out is not None and len(self.out) != len(self.tensors):
            raise ValueError("GradList: need one out tensor per gradient")
        if not self.tensors:
            raise ValueError("GradList: need at least one tensor")
        self.device = self.tensors[0].device if isinstance(self.tensors[0], torch.Tensor) else None
        n = len(self.tensors)
        kinds, numel = self._describe(self.tensors, "tensors")
        out_kinds, out_ptrs = None, None
        if self.out is not None:
            out_kinds, sizes = self._describe(self.out, "out")
            if sizes != numel:
                raise ValueError("GradList: out tensors need the gradients' sizes")
            out_kinds = (ctypes.c_int32 * n)(*out_kinds)
            out_ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.out])
        ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in self.tensors])
        sizes = (ctypes.c_int64 * n)(*numel)
        self.table = torch.empty(_size("qlora_gradlist_size", n, sizes), dtype=torch.uint8, device=self.device)
        self._struct = _GradListStruct()
        _check(_lib().qlora_gradlist_init(n, ptrs, (ctypes.c_int32 * n)(*kinds), sizes, out_ptrs, out_kinds,
                                          self.table.data_ptr() or None, self.table.numel(), ctypes.byref(self._struct),
                                          _raw_stream(self.table.get_device())), "gradlist_init")
        self._ref = ctypes.byref(self._struct)
        self._ws_bytes = _size("qlora_grad_workspace_size", self._ref)

    def _describe(self, tensors, name):
        index = self.device.index if self.device is not None else None
        kinds = [TYPES.get(t.dtype) if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == index
                 and t.is_contiguous() else None for t in tensors]
        if None in kinds:
            i = kinds.index(None)
            raise ValueError(f"{name}[{i}]: need a contiguous bfloat16 or float32 CUDA tensor on {self.device}")
        return kinds, [t.numel() for t in tensors]


def _grad_call(fn, grads, norm, ws, *args):
    if not isinstance(grads, GradList):
        raise ValueError("grads: need a GradList")
    dev = grads.device
    if norm is None:
        norm = torch.empty(1, dtype=_F32, device=dev)
    else:
        _tensors([(norm, _F32, "norm", (1,))], dev)
    st = _raw_stream(dev.index)
    ws = _workspace(ws, grads._ws_bytes, norm, dev.index, st)
    status = getattr(_lib(), fn)(grads._ref, *args, norm.data_ptr(), ws.data_ptr(), ws.numel(), st)
    if status:
        _check(status, fn[len("qlora_"):])
    return norm


def grad_norm(grads: GradList, norm: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """FP32 [1]: the square root of the sum of squares over all tensors of the list."""
    return _grad_call("qlora_grad_norm", grads, norm, ws)


def grad_clip(grads: GradList, max_norm: float, norm: torch.Tensor | None = None,
              ws: torch.Tensor | None = None) -> torch.Tensor:
    """Scales the list's gradients by min(1, max_norm / (norm + 1e-6)), into its out tensors or in
    place; returns the norm before clipping."""
    return _grad_call("qlora_grad_clip", grads, norm, ws, float(max_norm))


def adamw_step_clipped(master: torch.Tensor, m: torch.Tensor, v: torch.Tensor, grad: torch.Tensor,
                       norm: torch.Tensor, max_norm: float, step: int, lr: float, beta1: float = 0.9,
                       beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                       param: torch.Tensor | None = None) -> None:
    """adamw_step with grad scaled by min(1, max_norm / (norm + 1e-6)) as it is read; norm is the
    FP32 [1] tensor of grad_norm.  A norm that is not finite skips the step.  Slices of flat
    buffers start at multiples of four elements (16-byte aligned FP32, 8-byte aligned BF16)."""
    n = master.numel() if isinstance(master, torch.Tensor) else 0
    dev = master.device if isinstance(master, torch.Tensor) else None
    specs = [(t, torch.float32, name, getattr(t, "shape", None)) for t, name in ((master, "master"), (m, "m"), (v, "v"))]
    specs += [(grad, torch.bfloat16, "grad", getattr(grad, "shape", None)), (norm, torch.float32, "norm", (1,))]
    if param is not None:
        specs.append((param, torch.bfloat16, "param", getattr(param, "shape", None)))
    _tensors(specs, dev)
    if any(t.numel() != n for t in (m, v, grad)) or (param is not None and param.numel() != n):
        raise ValueError("adamw_step_clipped: all buffers need the same number of elements")
    _check(_lib().qlora_adamw_step_clipped(master.data_ptr(), m.data_ptr(), v.data_ptr(), grad.data_ptr(), _ptr(param),
                                           n, int(step), float(lr), float(beta1), float(beta2), float(eps),
                                           float(weight_decay), norm.data_ptr(), float(max_norm),
                                           _raw_stream(master.get_device())),
           "adamw_step_clipped")
