"""ctypes binding of include/qlora_train.h: block norms, the preference loss and gradient
clipping.  Argument marshalling only, as in ``_binding``: torch tensors provide device memory
and the stream, every step runs in the HIP library."""

from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _check, _check_ws, _ptr, _validate, _WS, load_library

TYPES = {torch.bfloat16: 0, torch.float32: 1}
NORM_MAX_WIDTH = 8192


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
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(t: torch.Tensor) -> int:
    return _raw_stream(t.get_device())


def _tensors(specs, device) -> None:
    """_validate, with a quick pass first."""
    if device is not None and device.type == "cuda":
        index = device.index
        for t, dtype, _, shape in specs:
            # (a tensor on the CPU has the device number -1)
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
                    and t.is_contiguous()):
                break
        else:
            return
    _validate(specs, device)


def _workspace(ws, nbytes: int, t: torch.Tensor, stream: int) -> torch.Tensor:
    """The caller's workspace, checked, or the binding's own for this device and stream."""
    if ws is not None:
        _check_ws(ws, t.device)
        return ws
    buf = _WS._bufs.get((t.get_device(), stream, "train"))
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
    M, d = x.shape
    dev = x.device
    specs = _norm_specs(x, y, w_post, gate, gate_rows, w_pre, M, d, "x")
    if x_out is not None:
        specs.append((x_out, x.dtype, "x_out", (M, d)))
    if h is not None:
        if not pre_norm:
            raise ValueError("h: given without pre_norm")
        specs.append((h, torch.bfloat16, "h", (M, d)))
    _tensors(specs, dev)
    if x_out is None:
        x_out = torch.empty_like(x)
    if pre_norm and h is None:
        h = torch.empty(M, d, dtype=torch.bfloat16, device=dev)
    _check(_lib().qlora_norm_residual_fwd(x.data_ptr(), _ptr(y), M, d, kind, int(post_norm), _ptr(w_post), _ptr(gate),
                                          int(gate_rows), _ptr(w_pre), res_scale, eps, x_out.data_ptr(), _ptr(h),
                                          _stream(x)), "norm_residual_fwd")
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
    M, d = stream.shape
    dev, bf16 = stream.device, torch.bfloat16
    specs = _norm_specs(x_out, y, w_post, gate, gate_rows, w_pre, M, d, "x_out")
    for t, dtype, name in ((dh, bf16, "dh"), (dx_out, stream.dtype, "dx_out"), (dx, stream.dtype, "dx"), (dy, bf16, "dy")):
        if t is not None:
            specs.append((t, dtype, name, (M, d)))
    _tensors(specs, dev)
    if dx is None:
        dx = torch.empty_like(stream)
    if y is not None and dy is None:
        dy = torch.empty_like(y)
    dw_post = torch.empty_like(w_post) if w_post is not None and need_weights else None
    dw_pre = torch.empty_like(w_pre) if w_pre is not None and need_weights else None
    dgate = torch.empty_like(gate) if gate is not None and need_gate else None
    rows = int(gate_rows) if gate is not None else 0
    st = _stream(stream)
    ws = _workspace(ws, norm_residual_workspace_size(M, d, rows), stream, st)
    _check(_lib().qlora_norm_residual_bwd(_ptr(x_out), _ptr(y), _ptr(dh), _ptr(dx_out), M, d, kind, int(post_norm),
                                          _ptr(w_post), _ptr(gate), rows, _ptr(w_pre), res_scale, eps, dx.data_ptr(),
                                          _ptr(dy), _ptr(dw_post), _ptr(dgate), _ptr(dw_pre), ws.data_ptr(),
                                          ws.numel(), st), "norm_residual_bwd")
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
        logps = torch.empty(lead, dtype=torch.float32, device=dev)
    st = _stream(logits)
    ws = _workspace(ws, logps_workspace_size(rows, V), logits, st)
    _check(_lib().qlora_token_logps(logits.data_ptr(), labels.data_ptr(), rows, V, kind, logps.data_ptr(),
                                    ws.data_ptr(), ws.numel(), st), "token_logps")
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
    specs = [(logits, logits.dtype, "logits", (n, S, V)), (labels, torch.int64, "labels", (n, S))]
    if ref_logps is not None:
        specs.append((ref_logps, torch.float32, "ref_logps", (n, S)))
    if dlogits is not None:
        if not need_grad:
            raise ValueError("dlogits: given with need_grad=False")
        specs.append((dlogits, logits.dtype, "dlogits", (n, S, V)))
    _tensors(specs, dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    log_ratios = torch.empty(n, dtype=torch.float32, device=dev)
    logps = torch.empty(n, S, dtype=torch.float32, device=dev)
    if need_grad and dlogits is None:
        dlogits = torch.empty_like(logits)
    st = _stream(logits)
    ws = _workspace(ws, preference_workspace_size(n // 2, S, V), logits, st)
    _check(_lib().qlora_preference_loss(logits.data_ptr(), labels.data_ptr(), _ptr(ref_logps), n // 2, S, V, kind,
                                        beta, label_smoothing, grad_scale, loss.data_ptr(), log_ratios.data_ptr(),
                                        logps.data_ptr(), _ptr(dlogits), ws.data_ptr(), ws.numel(), st), "preference_loss")
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
                                          _stream(self.table)), "gradlist_init")
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
        norm = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        _tensors([(norm, torch.float32, "norm", (1,))], dev)
    st = _stream(norm)
    ws = _workspace(ws, grads._ws_bytes, norm, st)
    _check(getattr(_lib(), fn)(grads._ref, *args, norm.data_ptr(), ws.data_ptr(), ws.numel(), st), fn[len("qlora_"):])
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
    FP32 [1] tensor of grad_norm.  A norm that is not finite skips the step."""
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
                                           float(weight_decay), norm.data_ptr(), float(max_norm), _stream(master)),
           "adamw_step_clipped")
