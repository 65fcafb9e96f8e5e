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
import struct
from typing import Optional, Sequence, Union

import torch

from . import _lib as L
from .binding import MatBatch, alloc_on

__all__ = [
    "int8_empty", "quantize_int8", "quantize_int8_workspace_bytes", "int8_matmul", "rms_norm", "rms_norm_backward",
    "rms_norm_backward_workspace_bytes", "distill_loss", "distill_loss_backward",
]

Tensors = Union[torch.Tensor, Sequence[torch.Tensor]]

_CODES = {torch.float32: L.OUO_F32, torch.bfloat16: L.OUO_BF16}

# One ouo_mat as bytes; a batch is their concatenation.  A call's descriptors
# live for the duration of the call.
_mat_bytes = struct.Struct("Pqqq").pack
_ptr_bytes = struct.Struct("P").pack
assert struct.calcsize("Pqqq") == ctypes.sizeof(L.OuoMat)

# The raw handle of a device's current stream: these calls take microseconds,
# and building a Stream object is one of them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _wrong_device(t: torch.Tensor, name: str, dev: int):
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    return ValueError(f"{name} is on {t.device}, the others on cuda:{dev}")


def _code(t: torch.Tensor, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _mat(t: torch.Tensor, name: str, dev: int, dtype: Optional[torch.dtype] = None) -> bytes:
    """A 2-D row-major tensor as an ouo_mat (its dtype as `dtype` says, or
    already looked up by _code)."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    r, c = shape
    ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError(f"{name} needs unit column stride")
    if ld < c:
        if r > 1:
            raise ValueError(f"{name}: rows overlap (stride {ld}, {c} columns)")
        ld = c
    if dev < 0 or t.get_device() != dev:
        raise _wrong_device(t, name, dev)
    return _mat_bytes(t.data_ptr(), r, c, ld)


def _vec(t: torch.Tensor, name: str, dev: int, n: int,
         dtype: Optional[torch.dtype] = torch.float32) -> int:
    """The address of a contiguous vector of at least n elements."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name} needs at least {n} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise _wrong_device(t, name, dev)
    return t.data_ptr()


def _mats(ts, name: str, dev: int, dtype: Optional[torch.dtype] = None) -> bytes:
    for t in ts:
        if t.dtype is not ts[0].dtype:
            raise TypeError(f"{name}: a batch must have one dtype")
    return b"".join([_mat(t, name, dev, dtype) for t in ts])


def _vecs(x: Tensors, name: str, dev: int, owners) -> bytes:
    """Pointers of one fp32 vector per matrix, one element per row."""
    ts = _list(x)
    if len(ts) != len(owners):
        raise ValueError(f"{name} needs one vector per matrix")
    return b"".join([_ptr_bytes(_vec(t, name, dev, m.shape[0])) for t, m in zip(ts, owners)])


def _scale(t: torch.Tensor, name: str, dev: int, rows: int) -> bytes:
    """_vecs of a single matrix."""
    if not isinstance(t, torch.Tensor):
        if len(t) != 1:
            raise ValueError(f"{name} needs one vector per matrix")
        t = t[0]
    return _ptr_bytes(_vec(t, name, dev, rows))


def _check_stream(stream, dev: int) -> None:
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")


def _workspace(need: int, given: Optional[torch.Tensor], dev: int, stream):
    """The caller's workspace, or one allocated here for the stream that uses
    it: (tensor or None, address, bytes)."""
    if need == 0:
        return None, None, 0
    if given is None:
        _check_stream(stream, dev)
        given = alloc_on(stream, need, torch.uint8, dev)
    return given, _vec(given, "workspace", dev, need, torch.uint8), given.numel()


_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_entry = {}


def _run(fname: str, dev: int, stream, *args) -> None:
    """Calls the library with the tensors' device current (the first one's,
    which every other was compared with), the stream last."""
    fn = _entry.get(fname)
    if fn is None:
        fn = _entry[fname] = getattr(L.lib(), fname)
    if stream is None:
        s = _raw_stream(dev)
    else:
        _check_stream(stream, dev)
        s = stream.cuda_stream
    if _get_device() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        L.check(fname, rc)


def _list(x: Tensors) -> Sequence[torch.Tensor]:
    if isinstance(x, torch.Tensor):
        return (x,)
    return x.tensors if isinstance(x, MatBatch) else x


def int8_empty(rows: int, cols: int, device=None) -> torch.Tensor:
    """An uninitialised rows x cols int8 matrix whose rows start on 16-byte
    boundaries (its row pitch is cols rounded up to 16), the layout that the
    tensor-core path of int8_matmul takes."""
    pitch = (cols + 15) // 16 * 16
    dev = "cuda" if device is None else device
    return torch.empty((rows, pitch), dtype=torch.int8, device=dev)[:, :cols]


def quantize_int8_workspace_bytes(X: Tensors, transpose: bool = False) -> int:
    xs = _list(X)
    if not xs:
        return 0
    return int(L.lib().quantize_int8_workspace_bytes(
        _mats(xs, "X", xs[0].get_device()), _code(xs[0], "X"), len(xs), 1 if transpose else 0))


def quantize_int8(X: Tensors, Q: Tensors, scale: Tensors, transpose: bool = False,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Q, scale <- X in 8 bits with one scale per row, or, with ``transpose``,
    X's transpose (one scale per column of X).  X, Q and scale are tensors, or
    lists of equal length.  Large transposed matrices take a workspace
    (allocated here unless given)."""
    if isinstance(X, torch.Tensor) and isinstance(Q, torch.Tensor):
        dev, code, n = X.get_device(), _code(X, "X"), 1
        x, q = _mat(X, "X", dev), _mat(Q, "Q", dev, torch.int8)
        sc = _scale(scale, "scale", dev, Q.shape[0])
    else:
        xs, qs = _list(X), _list(Q)
        n = len(xs)
        if len(qs) != n:
            raise ValueError(f"X has {n} matrices, Q {len(qs)}")
        if n == 0:
            return
        dev, code = xs[0].get_device(), _code(xs[0], "X")
        x, q = _mats(xs, "X", dev), _mats(qs, "Q", dev, torch.int8)
        sc = _vecs(scale, "scale", dev, qs)
    ws, wp, wn = None, None, 0  # ws: kept until the launch
    if transpose:
        ws, wp, wn = _workspace(L.lib().quantize_int8_workspace_bytes(x, code, n, 1), workspace,
                                dev, stream)
    _run("quantize_int8", dev, stream, x, code, q, sc, n, 1 if transpose else 0, wp, wn)


def int8_matmul(A: Tensors, a_scale: Tensors, B: Tensors, b_scale: Tensors, D: Tensors,
                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """D <- diag(a_scale) (A B^T) diag(b_scale), A (M x K) and B (N x K) 8-bit
    integers as quantize_int8 writes them.  Tensors, or lists of equal
    length.  Depths whose sums leave 32 bits go to int8_matmul_deep."""
    if isinstance(A, torch.Tensor) and isinstance(B, torch.Tensor) and isinstance(D, torch.Tensor):
        dev, n = A.get_device(), 1
        a, b = _mat(A, "A", dev, torch.int8), _mat(B, "B", dev, torch.int8)
        d, code = _mat(D, "D", dev), _code(D, "D")
        sa = _scale(a_scale, "a_scale", dev, A.shape[0])
        sb = _scale(b_scale, "b_scale", dev, B.shape[0])
        depth = A.shape[1]
    else:
        As, Bs, Ds = _list(A), _list(B), _list(D)
        n = len(As)
        if len(Bs) != n or len(Ds) != n:
            raise ValueError(f"A has {n} matrices, B {len(Bs)}, D {len(Ds)}")
        if n == 0:
            return
        dev = As[0].get_device()
        a, b = _mats(As, "A", dev, torch.int8), _mats(Bs, "B", dev, torch.int8)
        d, code = _mats(Ds, "D", dev), _code(Ds[0], "D")
        sa, sb = _vecs(a_scale, "a_scale", dev, As), _vecs(b_scale, "b_scale", dev, Bs)
        depth = max(t.shape[1] for t in As)
    st = None if status is None else _vec(status, "status", dev, 1, torch.int32)
    _run("int8_matmul" if depth <= L.OUO_INT8_MAX_DEPTH else "int8_matmul_deep", dev, stream, a, sa, b, sb, d, code, n, st)


def rms_norm(X: torch.Tensor, weight: torch.Tensor, Y: Optional[torch.Tensor] = None,
             Q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
             residual: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None,
             rstd: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None) -> None:
    """H <- X + residual; Y and / or (Q, scale in 8 bits) <- the norm of H
    times weight; rstd <- 1 / sqrt(mean(H^2) + eps) per row."""
    dev = X.get_device()
    x = _mat(X, "X", dev)
    rows, cols = X.shape
    r = h = y = q = sp = rp = None
    hc = yc = L.OUO_F32
    if H is not None:
        h, hc = _mat(H, "H", dev), _code(H, "H")
    if residual is not None:
        if H is not None and H.dtype is not residual.dtype:
            raise TypeError("residual and H must have one dtype")
        r = _mat(residual, "residual", dev)
    if Y is not None:
        y, yc = _mat(Y, "Y", dev), _code(Y, "Y")
    if Q is not None:
        if scale is None:
            raise ValueError("Q needs scale")
        q, sp = _mat(Q, "Q", dev, torch.int8), _vec(scale, "scale", dev, rows)
    if rstd is not None:
        rp = _vec(rstd, "rstd", dev, rows)
    _run("rms_norm", dev, stream, x, _code(X, "X"), r, h, hc, _weight(weight, dev, cols),
         _code(weight, "weight"), eps, y, yc, q, sp, rp)


def _weight(weight: torch.Tensor, dev: int, cols: int) -> int:
    if weight.numel() != cols:
        raise ValueError(f"weight has {weight.numel()} elements, the rows {cols}")
    return _vec(weight, "weight", dev, cols, None)


def rms_norm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return int(L.lib().rms_norm_backward_workspace_bytes(rows, cols))


def rms_norm_backward(dY: torch.Tensor, H: torch.Tensor, weight: torch.Tensor,
                      rstd: torch.Tensor, dX: torch.Tensor,
                      dweight: Optional[torch.Tensor] = None,
                      dH: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """dX <- dH + the gradient of rms_norm's H; dweight <- that of its
    weight."""
    dev = dY.get_device()
    dy, h, dx = _mat(dY, "dY", dev), _mat(H, "H", dev), _mat(dX, "dX", dev)
    rows, cols = dY.shape
    w, rp = _weight(weight, dev, cols), _vec(rstd, "rstd", dev, rows)
    dh = dwp = ws = wp = None  # ws: kept until the launch
    wn = 0
    if dH is not None:
        if dH.dtype is not dX.dtype:
            raise TypeError("dH and dX must have one dtype")
        dh = _mat(dH, "dH", dev)
    if dweight is not None:
        dwp = _vec(dweight, "dweight", dev, cols)
        ws, wp, wn = _workspace(rms_norm_backward_workspace_bytes(rows, cols), workspace, dev,
                                stream)
    _run("rms_norm_backward", dev, stream, dy, _code(dY, "dY"), h, _code(H, "H"), w,
         _code(weight, "weight"), rp, dh, dx, _code(dX, "dX"), dwp, wp, wn)


def distill_loss(S: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor, loss: torch.Tensor,
                 lse: torch.Tensor, temperature: float = 1.0, stream=None) -> None:
    """loss <- tau^2 KL(softmax(teacher / tau) || softmax(S / tau) at idx) per
    row; lse <- the log of the student's normalizer."""
    dev = S.get_device()
    s, t, i = _mat(S, "S", dev), _mat(teacher, "teacher", dev), _mat(idx, "idx", dev, torch.int32)
    rows = S.shape[0]
    _run("distill_loss", dev, stream, s, _code(S, "S"), t, _code(teacher, "teacher"), i,
         temperature, _vec(loss, "loss", dev, rows), _vec(lse, "lse", dev, rows))


def distill_loss_backward(S: torch.Tensor, teacher: torch.Tensor, idx: torch.Tensor,
                          lse: torch.Tensor, dloss: torch.Tensor, dS: torch.Tensor,
                          temperature: float = 1.0, stream=None) -> None:
    """dS <- the gradient of sum_t dloss_t loss_t with respect to S."""
    dev = S.get_device()
    s, t, i = _mat(S, "S", dev), _mat(teacher, "teacher", dev), _mat(idx, "idx", dev, torch.int32)
    rows = S.shape[0]
    _run("distill_loss_backward", dev, stream, s, _code(S, "S"), t, _code(teacher, "teacher"), i,
         temperature, _vec(lse, "lse", dev, rows), _vec(dloss, "dloss", dev, rows),
         _mat(dS, "dS", dev), _code(dS, "dS"))
