"""Binding of the token-matrix operators of liborthoupd.so: 8-bit products,
root-mean-square norm, distillation loss.

They make the gradients that the optimizer step consumes and read the weights
that it writes.  As in ``binding``, each function marshals tensors into the C
entry point of the same name (``include/orthoupd.h`` documents them), checks
what the library cannot see (types, devices, strides) and raises ``OuoError``
on a nonzero return.  Outputs are the caller's tensors; everything is
asynchronous on the current stream of the tensors' device (or ``stream=``).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Union

import torch

from . import _lib as L

__all__ = [
    "int8_empty", "quantize_int8", "int8_matmul", "rms_norm", "rms_norm_backward",
    "rms_norm_backward_workspace_bytes", "distill_loss", "distill_loss_backward",
]

Tensors = Union[torch.Tensor, Sequence[torch.Tensor]]

_CODES = {torch.float32: L.OUO_F32, torch.bfloat16: L.OUO_BF16}


class _Call:
    """The device and stream of one call: every tensor has to be on the
    first one's device."""

    __slots__ = ("dev",)

    def __init__(self):
        self.dev = -1

    def on(self, t: torch.Tensor, name: str) -> None:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        d = t.get_device()
        if self.dev < 0:
            self.dev = d
        elif d != self.dev:
            raise ValueError(f"{name} is on cuda:{d}, the others on cuda:{self.dev}")

    def mat(self, t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None) -> L.OuoMat:
        if dtype is None:
            if t.dtype not in _CODES:
                raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
        elif t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
        r, c = t.shape
        ld, one = t.stride()
        if c > 1 and one != 1:
            raise ValueError(f"{name} needs unit column stride")
        if ld < c:
            if r > 1 and c > 0:
                raise ValueError(f"{name}: rows overlap (stride {ld}, {c} columns)")
            ld = c
        self.on(t, name)
        return L.OuoMat(t.data_ptr(), r, c, ld)

    def vec(self, t: torch.Tensor, name: str, n: int,
            dtype: Optional[torch.dtype] = torch.float32) -> int:
        if dtype is None:
            if t.dtype not in _CODES:
                raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
        elif t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.numel() < n:
            raise ValueError(f"{name} needs at least {n} elements, got {t.numel()}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        self.on(t, name)
        return t.data_ptr()

    def run(self, fname: str, stream, *args) -> None:
        """Calls the library with this device current and the stream last."""
        if stream is None:
            s = torch.cuda.current_stream(self.dev)
        else:
            s = stream
            if s.device.index != self.dev:
                raise ValueError(f"the stream is on {s.device}, the tensors on cuda:{self.dev}")
        fn = getattr(L.lib(), fname)
        if torch.cuda.current_device() == self.dev:
            rc = fn(*args, s.cuda_stream)
        else:
            with torch.cuda.device(self.dev):
                rc = fn(*args, s.cuda_stream)
        if rc:
            L.check(fname, rc)


def _list(x: Tensors) -> Sequence[torch.Tensor]:
    return (x,) if isinstance(x, torch.Tensor) else x


def _mats(call: _Call, ts, name: str, dtype=None):
    arr = (L.OuoMat * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = call.mat(t, name, dtype)
        if t.dtype != ts[0].dtype:
            raise TypeError(f"{name}: a batch must have one dtype")
    return arr


def _vecs(call: _Call, ts, name: str, counts):
    if len(ts) != len(counts):
        raise ValueError(f"{name} needs one vector per matrix")
    arr = (ctypes.c_void_p * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = call.vec(t, name, counts[i])
    return arr


def int8_empty(rows: int, cols: int, device=None) -> torch.Tensor:
    """An uninitialised rows x cols int8 matrix whose rows start on 16-byte
    boundaries (its row pitch is cols rounded up to 16), the layout that the
    tensor-core path of int8_matmul takes."""
    pitch = (cols + 15) // 16 * 16
    dev = "cuda" if device is None else device
    return torch.empty((rows, pitch), dtype=torch.int8, device=dev)[:, :cols]


def quantize_int8(X: Tensors, Q: Tensors, scale: Tensors, transpose: bool = False,
                  stream=None) -> None:
    """Q, scale <- X in 8 bits with one scale per row, or, with ``transpose``,
    X's transpose (one scale per column of X).  X, Q and scale are tensors, or
    lists of equal length."""
    xs, qs, ss = _list(X), _list(Q), _list(scale)
    n = len(xs)
    if len(qs) != n:
        raise ValueError(f"X has {n} matrices, Q {len(qs)}")
    if n == 0:
        return
    c = _Call()
    xa, qa = _mats(c, xs, "X"), _mats(c, qs, "Q", torch.int8)
    sa = _vecs(c, ss, "scale", [q.shape[0] for q in qs])
    c.run("quantize_int8", stream, xa, _CODES[xs[0].dtype], qa, sa, n, 1 if transpose else 0)


def int8_matmul(A: Tensors, a_scale: Tensors, B: Tensors, b_scale: Tensors, D: Tensors,
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """D <- diag(a_scale) (A B^T) diag(b_scale), A (M x K) and B (N x K) 8-bit
    integers as quantize_int8 writes them.  Tensors, or lists of equal
    length."""
    As, Bs, Ds = _list(A), _list(B), _list(D)
    n = len(As)
    if len(Bs) != n or len(Ds) != n:
        raise ValueError(f"A has {n} matrices, B {len(Bs)}, D {len(Ds)}")
    if n == 0:
        return
    c = _Call()
    aa, ba = _mats(c, As, "A", torch.int8), _mats(c, Bs, "B", torch.int8)
    da = _mats(c, Ds, "D")
    sa = _vecs(c, _list(a_scale), "a_scale", [t.shape[0] for t in As])
    sb = _vecs(c, _list(b_scale), "b_scale", [t.shape[0] for t in Bs])
    st = None if status is None else c.vec(status, "status", 1, torch.int32)
    c.run("int8_matmul", stream, aa, sa, ba, sb, da, _CODES[Ds[0].dtype], n, st)


def _ref(m: Optional[L.OuoMat]):
    return None if m is None else ctypes.byref(m)


def rms_norm(X: torch.Tensor, weight: torch.Tensor, Y: Optional[torch.Tensor] = None,
             Q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None,
             rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    """H <- X + residual; Y and / or (Q, scale in 8 bits) <- the norm of H
    times weight; rstd <- 1 / sqrt(mean(H^2) + eps) per row."""
    c = _Call()
    x = c.mat(X, "X")
    rows, cols = X.shape
    w = c.vec(weight, "weight", cols, None)
    if weight.numel() != cols:
        raise ValueError(f"weight has {weight.numel()} elements, X {cols} columns")
    r = h = y = q = sp = rp = None
    if residual is not None:
        r = c.mat(residual, "residual")
        if H is not None and H.dtype != residual.dtype:
            raise TypeError("residual and H must have one dtype")
    if H is not None:
        h = c.mat(H, "H")
    if Y is not None:
        y = c.mat(Y, "Y")
    if Q is not None:
        q = c.mat(Q, "Q", torch.int8)
        if scale is None:
            raise ValueError("Q needs scale")
        sp = c.vec(scale, "scale", rows)
    if rstd is not None:
        rp = c.vec(rstd, "rstd", rows)
    c.run("rms_norm", stream, ctypes.byref(x), _CODES[X.dtype], _ref(r), _ref(h),
          L.OUO_F32 if H is None else _CODES[H.dtype], w, _CODES[weight.dtype], eps, _ref(y),
          L.OUO_F32 if Y is None else _CODES[Y.dtype], _ref(q), sp, rp)


def rms_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(L.lib().rms_norm_backward_workspace_bytes(rows, cols))


def rms_norm_backward(dY: torch.Tensor, H: torch.Tensor, weight: torch.Tensor,
                      rstd: torch.Tensor, dX: torch.Tensor,
                      dweight: Optional[torch.Tensor] = None,
                      dH: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dX <- dH + the gradient of rms_norm's H; dweight <- that of its
    weight."""
    c = _Call()
    dy, h, dx = c.mat(dY, "dY"), c.mat(H, "H"), c.mat(dX, "dX")
    rows, cols = dY.shape
    w = c.vec(weight, "weight", cols, None)
    if weight.numel() != cols:
        raise ValueError(f"weight has {weight.numel()} elements, dY {cols} columns")
    rp = c.vec(rstd, "rstd", rows)
    dh = dwp = wp = None
    wn = 0
    if dH is not None:
        if dH.dtype != dX.dtype:
            raise TypeError("dH and dX must have one dtype")
        dh = c.mat(dH, "dH")
    if dweight is not None:
        dwp = c.vec(dweight, "dweight", cols)
        need = rms_norm_backward_workspace_bytes(rows, cols)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dY.device)
            if stream is not None:
                workspace.record_stream(stream)
        wp, wn = c.vec(workspace, "workspace", need, torch.uint8), workspace.numel()
    c.run("rms_norm_backward", stream, ctypes.byref(dy), _CODES[dY.dtype], ctypes.byref(h),
          _CODES[H.dtype], w, _CODES[weight.dtype], rp, _ref(dh), ctypes.byref(dx),
          _CODES[dX.dtype], dwp, wp, wn)


def _teacher(c: _Call, S, teacher, idx):
    return c.mat(S, "S"), c.mat(teacher, "teacher"), c.mat(idx, "idx", torch.int32)


def distill_loss(S: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor, loss: torch.Tensor,
                 lse: torch.Tensor, temperature: float = 1.0, stream=None) -> None:
    """loss <- tau^2 KL(softmax(teacher / tau) || softmax(S / tau) at idx) per
    row; lse <- the log of the student's normalizer."""
    c = _Call()
    s, t, i = _teacher(c, S, teacher, idx)
    rows = S.shape[0]
    lp, ep = c.vec(loss, "loss", rows), c.vec(lse, "lse", rows)
    c.run("distill_loss", stream, ctypes.byref(s), _CODES[S.dtype], ctypes.byref(t),
          _CODES[teacher.dtype], ctypes.byref(i), temperature, lp, ep)


def distill_loss_backward(S: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor,
                          lse: torch.Tensor, dloss: torch.Tensor, dS: torch.Tensor,
                          temperature: float = 1.0, stream=None) -> None:
    """dS <- the gradient of sum_t dloss_t loss_t with respect to S."""
    c = _Call()
    s, t, i = _teacher(c, S, teacher, idx)
    rows = S.shape[0]
    ep, gp = c.vec(lse, "lse", rows), c.vec(dloss, "dloss", rows)
    d = c.mat(dS, "dS")
    c.run("distill_loss_backward", stream, ctypes.byref(s), _CODES[S.dtype], ctypes.byref(t),
          _CODES[teacher.dtype], ctypes.byref(i), temperature, ep, gp, ctypes.byref(d),
          _CODES[dS.dtype])
