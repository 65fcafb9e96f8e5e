"""CPU checks of what the token-matrix calls refuse, in the library and in
the binding; nothing is launched (the pointers are fake)."""
import ctypes

import pytest
import torch

import orthonormalized_update_optimizers_b200 as ouo
from orthonormalized_update_optimizers_b200 import _lib as L
from orthonormalized_update_optimizers_b200 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def _m(rows, cols, ptr=0x10000, ld=None):
    return (L.OuoMat * 1)(L.OuoMat(ptr, rows, cols, cols if ld is None else ld))


def _v(ptr=0x20000):
    return (ctypes.c_void_p * 1)(ptr)


BAD, UNSUP, WS, NODEV = -1, -2, -3, -5


def _quant(lib, x=None, q=None, s=None, dt=L.OUO_BF16, t=0, n=1):
    return lib.quantize_int8(_m(4, 8) if x is None else x, dt, _m(4, 8) if q is None else q,
                             _v() if s is None else s, n, t, None, 0, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=_m(4, 8, None)), b"NULL"), (dict(x=_m(4, 8, 0x10001)), b"aligned"),
    (dict(x=_m(4, 8, ld=7)), b"ld"), (dict(q=_m(4, 7)), b"needs 4 x 8"),
    (dict(t=1), b"needs 8 x 4"), (dict(t=2), b"transpose"), (dict(dt=2), b"dtype"),
    (dict(s=_v(None)), b"NULL"), (dict(s=_v(0x20002)), b"aligned"), (dict(n=-1), b"nmat"),
    (dict(n=4097), b"nmat"), (dict(x=_m(-1, 8)), b"negative"),
    (dict(x=_m((1 << 30) + 1, 8), q=_m((1 << 30) + 1, 8)), b"large"),
])
def test_quantize_refuses(lib, kw, msg):
    assert _quant(lib, **kw) == BAD and msg in lib.ouo_last_error()
    assert lib.quantize_int8(_m(1, 1), 0, _m(1, 1), None, 1, 0, None, 0, None) == BAD


def test_quantize_workspace(lib):
    big, out = _m(8192, 4096), _m(4096, 8192, 0x90000)
    need = lib.quantize_int8_workspace_bytes(big, L.OUO_BF16, 1, 1)
    assert need >= 4096 * 4 and lib.quantize_int8_workspace_bytes(big, L.OUO_BF16, 1, 0) == 0
    assert lib.quantize_int8_workspace_bytes(_m(16, 64), L.OUO_BF16, 1, 1) == 0
    for ws, n in ((None, need), (0x60000, need - 1), (0x60008, need)):
        assert lib.quantize_int8(big, L.OUO_BF16, out, _v(), 1, 1, ws, n, None) == WS
        assert b"workspace" in lib.ouo_last_error()


def _mm(lib, a=None, b=None, d=None, sa=None, sb=None, dt=L.OUO_BF16, st=None):
    return lib.int8_matmul(_m(4, 32) if a is None else a, _v() if sa is None else sa,
                           _m(6, 32) if b is None else b, _v() if sb is None else sb,
                           _m(4, 6) if d is None else d, dt, 1, st, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(b=_m(6, 31)), BAD, b"columns"), (dict(d=_m(6, 4)), BAD, b"needs 4 x 6"),
    (dict(sa=_v(None)), BAD, b"a_scale"), (dict(sb=_v(0x3)), BAD, b"b_scale"),
    (dict(dt=2), BAD, b"dtype"), (dict(st=0x3), BAD, b"dev_status"),
    (dict(a=_m(4, 131072), b=_m(6, 131072)), UNSUP, b"32 bits"),
    (dict(a=_m(4, 32, None)), BAD, b"NULL"), (dict(d=_m(4, 6, 0x10001)), BAD, b"aligned"),
])
def test_matmul_refuses(lib, kw, code, msg):
    assert _mm(lib, **kw) == code and msg in lib.ouo_last_error()


def _ref(m):
    return None if m is None else ctypes.byref(m[0])


def _rms(lib, x=_m(4, 8), r=None, h=None, w=0x30000, eps=1e-6, y=_m(4, 8), q=None, s=None,
         xd=1, hd=1, wd=1, yd=1, rstd=None):
    return lib.rms_norm(_ref(x), xd, _ref(r), _ref(h), hd, w, wd, eps, _ref(y), yd, _ref(q), s,
                        rstd, None)


@pytest.mark.parametrize("kw,msg", [
    (dict(x=None), b"X"), (dict(y=None), b"required"), (dict(r=_m(4, 8)), b"H"),
    (dict(h=_m(4, 9)), b"needs 4 x 8"), (dict(r=_m(3, 8), h=_m(4, 8)), b"residual"),
    (dict(w=None), b"weight"), (dict(w=0x30001), b"weight"), (dict(eps=-1.0), b"eps"),
    (dict(eps=float("nan")), b"eps"), (dict(q=_m(4, 8)), b"scale"), (dict(q=_m(8, 4), s=4), b"Q"),
    (dict(xd=2), b"dtype"), (dict(wd=3), b"dtype"), (dict(yd=2), b"dtype"),
    (dict(h=_m(4, 8), hd=5), b"dtype"), (dict(rstd=2), b"rstd"),
    (dict(x=_m(4, 0), y=_m(4, 0)), b"columns"),
])
def test_rms_norm_refuses(lib, kw, msg):
    assert _rms(lib, **kw) == BAD and msg in lib.ouo_last_error()


# large enough to need a workspace
_BIG = dict(dy=_m(64, 4096), h=_m(64, 4096, 0x70000), dx=_m(64, 4096, 0x80000))


def _rmsb(lib, dy=_m(4, 8), h=_m(4, 8), w=0x30000, rstd=0x40000, dh=None, dx=_m(4, 8), dw=0x50000,
          ws=0x60000, wn=1 << 20, dxd=1):
    return lib.rms_norm_backward(_ref(dy), 1, _ref(h), 1, w, 1, rstd, _ref(dh), _ref(dx), dxd, dw,
                                 ws, wn, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dy=None), BAD, b"required"), (dict(h=_m(4, 7)), BAD, b"H"),
    (dict(dx=_m(5, 8)), BAD, b"dX"), (dict(dh=_m(4, 9)), BAD, b"dH"),
    (dict(rstd=None), BAD, b"rstd"), (dict(w=None), BAD, b"weight"), (dict(dxd=2), BAD, b"dtype"),
    (dict(_BIG, ws=None), WS, b"workspace"), (dict(_BIG, wn=16), WS, b"workspace"),
    (dict(_BIG, ws=0x60004), WS, b"aligned"), (dict(dw=2), BAD, b"dweight"),
])
def test_rms_norm_backward_refuses(lib, kw, code, msg):
    assert _rmsb(lib, **kw) == code and msg in lib.ouo_last_error()


def test_rms_workspace_query(lib):
    assert ouo.rms_norm_backward_workspace_bytes(0, 64) == 0
    assert ouo.rms_norm_backward_workspace_bytes(1, 64) == 0  # a few tokens need none
    assert ouo.rms_norm_backward_workspace_bytes(64, 4096) >= 4096 * 4
    assert ouo.rms_norm_backward_workspace_bytes(1 << 20, 64) < 1 << 20
    assert ouo.rms_norm_backward_workspace_bytes(-1, 64) == 0


def _kd(lib, s=_m(4, 50), t=_m(4, 6), i=_m(4, 6), tau=1.0, loss=0x30000, lse=0x40000, sd=1, td=0):
    return lib.distill_loss(_ref(s), sd, _ref(t), td, _ref(i), tau, loss, lse, None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(s=None), BAD, b"required"), (dict(i=_m(4, 5)), BAD, b"idx"),
    (dict(t=_m(3, 6)), BAD, b"teacher"), (dict(t=_m(4, 0), i=_m(4, 0)), BAD, b"entries"),
    (dict(t=_m(4, 1025), i=_m(4, 1025)), UNSUP, b"1024"), (dict(tau=0.0), BAD, b"temperature"),
    (dict(tau=float("nan")), BAD, b"temperature"), (dict(loss=None), BAD, b"loss"),
    (dict(lse=0x40001), BAD, b"lse"), (dict(sd=2), BAD, b"dtype"), (dict(td=2), BAD, b"dtype"),
    (dict(s=_m(4, 0)), BAD, b"columns"), (dict(i=_m(4, 6, 0x10002)), BAD, b"aligned"),
])
def test_distill_refuses(lib, kw, code, msg):
    assert _kd(lib, **kw) == code and msg in lib.ouo_last_error()
    kw = {k: v for k, v in kw.items() if k not in ("loss",)}
    args = dict(s=_m(4, 50), t=_m(4, 6), i=_m(4, 6), tau=1.0, lse=0x40000, sd=1, td=0)
    args.update(kw)
    rc = lib.distill_loss_backward(_ref(args["s"]), args["sd"], _ref(args["t"]), args["td"],
                                   _ref(args["i"]), args["tau"], args["lse"], 0x50000,
                                   _ref(args["s"]), 1, None)
    if kw:
        assert rc == code


def test_distill_backward_refuses_what_is_not_in_place(lib):
    s, o, t = _m(4, 50), _m(4, 50, ld=64), _m(4, 6, 0x90000)
    call = lib.distill_loss_backward
    assert call(_ref(s), 1, _ref(t), 0, _ref(t), 1.0, 0x100, 0x200, _ref(o), 1, None) == BAD
    assert call(_ref(s), 1, _ref(t), 0, _ref(t), 1.0, 0x100, 0x200, _ref(s), 0, None) == BAD
    assert b"in place" in lib.ouo_last_error()
    assert call(_ref(s), 1, _ref(t), 0, _ref(t), 1.0, 0x100, 0x200, None, 1, None) == BAD
    assert call(_ref(s), 1, _ref(t), 0, _ref(t), 1.0, 0x100, None, _ref(s), 1, None) == BAD


def test_in_place_needs_the_same_layout(lib):
    x, wide = _m(4, 8), _m(4, 8, ld=16)
    assert _rms(lib, x=x, h=wide) == BAD and b"H and X" in lib.ouo_last_error()
    assert _rms(lib, x=x, h=x, hd=0) == BAD and b"H and X" in lib.ouo_last_error()
    o = _m(4, 8, 0x90000)
    assert _rms(lib, x=o, r=x, h=wide) == BAD and b"H and residual" in lib.ouo_last_error()
    assert _rmsb(lib, dy=x, dx=wide) == BAD and b"dX and dY" in lib.ouo_last_error()
    assert _rmsb(lib, dy=x, dx=x, dxd=0) == BAD and b"dX and dY" in lib.ouo_last_error()
    assert _rmsb(lib, dy=o, dx=x, dh=wide) == BAD and b"dX and dH" in lib.ouo_last_error()


def test_without_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _quant(lib) == NODEV and _mm(lib) == NODEV and _rms(lib) == NODEV
    assert _rmsb(lib) == NODEV and _kd(lib) == NODEV


@pytest.mark.parametrize("call", [
    lambda x: ouo.quantize_int8(x, x.to(torch.int8), x[0]),
    lambda x: ouo.int8_matmul(x.to(torch.int8), x[0], x.to(torch.int8), x[0], x),
    lambda x: ouo.rms_norm(x, x[0], Y=x),
    lambda x: ouo.rms_norm_backward(x, x, x[0], x[:, 0], x),
    lambda x: ouo.distill_loss(x, x, x.int(), x[0], x[0]),
    lambda x: ouo.distill_loss_backward(x, x, x.int(), x[0], x[0], x),
])
def test_binding_refuses_host_tensors(call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(torch.zeros(4, 4))


def test_binding_refuses_types_and_layouts():
    x = torch.zeros(4, 4)
    with pytest.raises(TypeError, match="int8"):
        ouo.int8_matmul(x, x[0], x, x[0], x)
    with pytest.raises(TypeError, match="unsupported dtype"):
        ouo.quantize_int8(x.half(), x.to(torch.int8), x[0])
    with pytest.raises(ValueError, match="2-D"):
        ouo.rms_norm(x[0], x[0], Y=x)
    with pytest.raises(ValueError, match="unit column stride"):
        ouo.rms_norm(torch.zeros(4, 5).t(), x[0], Y=x)
    with pytest.raises(ValueError, match="overlap"):
        ouo.rms_norm(x[:1].expand(4, 4), x[0], Y=x)
    with pytest.raises(ValueError, match="2 matrices"):
        ouo.quantize_int8([x, x], [x], x[0])
    ouo.quantize_int8([], [], [])
    ouo.int8_matmul([], [], [], [], [])
