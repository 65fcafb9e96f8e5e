"""GPU parity of the token-matrix operators (8-bit quantization and product,
norm, distillation loss) against the float64 oracle: odd sizes, strides,
masks, empty rows, in-place forms, streams and graphs.

Tolerances count roundings: U32 = 2^-24 is half a step of fp32, UOUT that of
the output's type.  A sum of n terms in the kernels' order (runs of at most
`run` terms per thread, then a tree) is off by at most (run + 32) U32 times the
sum of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import orthonormalized_update_optimizers_b200 as ouo
from oracle import tokens as ot

from ._util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U32 = 2.0 ** -24
UOUT = {BF: 2.0 ** -8, F32: U32}


def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


class Guard:
    """A rows x cols view of a larger buffer (row pitch, offset in elements)
    whose other bytes must stay as they were."""

    def __init__(self, rows, cols, dtype, pad=0, off=0, fill=None):
        pitch = cols + pad
        n = off + (rows + 1) * pitch + 8
        self.buf = torch.full((n,), 77, device=DEV).to(dtype)
        self.v = self.buf[off:off + rows * pitch].view(rows, pitch)[:, :cols]
        if fill is not None:
            self.v.copy_(fill)
        self.mask = torch.ones(n, dtype=torch.bool, device=DEV)
        self.mask[off:off + rows * pitch].view(rows, pitch)[:, :cols] = False

    def check(self):
        assert bool((self.buf[self.mask].float() == 77).all()), "written outside the matrix"


# ---------------------------------------------------------- quantize_int8


def _check_quant(q, scale, x):
    """q and scale against x (float64, rows = rows of q)."""
    qe, se = ot.quantize(x)
    # amax is exact; amax / 127 is rounded once (in fp32's denormals to a
    # half step of 2^-149)
    assert np.all(np.abs(scale - se) <= 2 * U32 * se + 2.0 ** -150)
    # q = rint(x * fl(127 / amax)): two roundings of a value up to 127
    # (three with the scaling by a power of two, which is exact)
    assert np.all(np.abs(q - qe) <= 0.5 + 127 * 4 * U32)
    assert q.min(initial=0) >= -127 and q.max(initial=0) <= 127


SHAPES = [(1, 1), (1, 4096), (3, 7), (33, 70), (5, 129), (64, 256), (130, 1000), (2, 20000),
          (257, 31), (4100, 65)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("layout", ["tight", "pitch", "odd"])
def test_quantize(dtype, transpose, layout):
    xs, qs, ss = [], [], []
    pad, off = {"tight": (0, 0), "pitch": (24, 0), "odd": (3, 1)}[layout]
    for i, (m, n) in enumerate(SHAPES):
        x = torch.randn((m, n), generator=_rng(i), device=DEV) * 10.0 ** (i - 4)
        x = x.to(dtype)
        if m > 2:
            x[1] = 0
            x[0, n // 2] *= 50
        xs.append(Guard(m, n, dtype, pad, off, x).v)
        a, b = (n, m) if transpose else (m, n)
        qs.append(Guard(a, b, torch.int8, pad, off))
        ss.append(torch.full((a + 1,), 77.0, device=DEV))
    keep = [x.clone() for x in xs]
    ouo.quantize_int8(xs, [q.v for q in qs], ss, transpose=transpose)
    torch.cuda.synchronize()
    for x, k, q, s in zip(xs, keep, qs, ss):
        assert torch.equal(x, k)
        q.check()
        assert s[-1] == 77
        x64 = to64(x).T if transpose else to64(x)
        _check_quant(q.v.cpu().numpy().astype(np.float64), to64(s[:-1]), x64)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,off", [
    (2048, 1024, 0, 0), (1100, 2049, 0, 0), (4097, 1000, 8, 0), (300, 9000, 3, 1),
    (20001, 130, 6, 0), (60, 40000, 0, 0), (40000, 5, 0, 0), (30000, 32, 0, 0)])
def test_quantize_large_transposed(rows, cols, pad, off, dtype):
    x = torch.randn((rows, cols), generator=_rng(rows), device=DEV)
    x[rows // 2] *= 30
    x[:, 3] = 0
    x[5, 4] = float("nan")
    x = Guard(rows, cols, dtype, pad, off, x)
    q, s = Guard(cols, rows, torch.int8, pad, off), torch.full((cols + 1,), 77.0, device=DEV)
    ouo.quantize_int8(x.v, q.v, s, transpose=True)
    q.check()
    x.check()
    assert s[-1] == 77 and torch.isnan(s[4]) and not q.v[4].any()
    ok = np.arange(cols) != 4
    _check_quant(to64(q.v)[ok], to64(s[:-1])[ok], to64(x.v).T[ok])


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_extremes(transpose):
    big, tiny = torch.finfo(F32).max, 2.0 ** -140
    rows = [[0.0, 0, 0, 0], [1, float("nan"), 2, 3], [1, float("inf"), 2, 3],
            [-float("inf"), 1, 1, 1], [big, -big, big / 2, 1], [tiny, -tiny, tiny / 2, 0],
            [2.0 ** -97, 2.0 ** -98, 0, -2.0 ** -99], [-0.0, 0.0, 0, 0], [5, 5, -5, 5]]
    x = torch.tensor(rows, device=DEV)
    r = x.t().contiguous() if transpose else x
    q, s = torch.empty((9, 4), dtype=torch.int8, device=DEV), torch.empty(9, device=DEV)
    ouo.quantize_int8(r, q, s, transpose=transpose)
    q, s = q.cpu(), s.cpu()
    for i in (1, 2, 3):
        assert torch.isnan(s[i]) and not q[i].any()
    ok = [0, 4, 5, 6, 7, 8]
    _check_quant(q[ok].numpy().astype(np.float64), to64(s[ok]), to64(x)[ok])


def test_quantize_empty():
    s = torch.full((4,), 77.0, device=DEV)
    ouo.quantize_int8(torch.empty((0, 8), device=DEV), ouo.int8_empty(0, 8), s)
    assert (s == 77).all()
    ouo.quantize_int8(torch.empty((0, 4), device=DEV), ouo.int8_empty(4, 0), s, transpose=True)
    assert (s == 0).all()
    s.fill_(77)
    ouo.quantize_int8(torch.empty((4, 0), device=DEV), ouo.int8_empty(4, 0), s)
    assert (s == 0).all()


@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_batch_with_empty_matrices(transpose):
    shapes = [(0, 8), (5, 16), (3, 0), (0, 0), (7, 9), (0, 4)]
    xs = [torch.randn(s, generator=_rng(i), device=DEV) for i, s in enumerate(shapes)]
    qs = [ouo.int8_empty(n, m) if transpose else ouo.int8_empty(m, n) for m, n in shapes]
    ss = [torch.full((q.shape[0] + 1,), 77.0, device=DEV) for q in qs]
    ouo.quantize_int8(xs, qs, ss, transpose=transpose)
    for x, q, s in zip(xs, qs, ss):
        assert s[-1] == 77
        if x.numel():
            _check_quant(to64(q), to64(s[:-1]), to64(x).T if transpose else to64(x))
        else:
            assert (s[:-1] == 0).all()


def test_quantize_many_matrices():
    """More matrices than one launch's table holds."""
    xs = [torch.randn((1 + i % 5, 1 + i % 37), generator=_rng(i), device=DEV) for i in range(300)]
    qs = [ouo.int8_empty(*x.shape) for x in xs]
    ss = [torch.empty(x.shape[0], device=DEV) for x in xs]
    ouo.quantize_int8(xs, qs, ss)
    for x, q, s in zip(xs, qs, ss):
        _check_quant(q.cpu().numpy().astype(np.float64), to64(s), to64(x))


# ------------------------------------------------------------ int8_matmul


def _ints(shape, seed, lo=-127, hi=127):
    return torch.randint(lo, hi + 1, shape, generator=_rng(seed), device=DEV, dtype=torch.int8)


def _check_mm(d, a, sa, b, sb):
    e = ot.int8_matmul(a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy())
    got = to64(d)
    # int -> fp32, two products, the output's rounding
    tol = (1 + UOUT[d.dtype]) * (1 + U32) ** 3 - 1
    assert np.all(np.abs(got - e) <= tol * np.abs(e))


MM = [(1, 1, 1), (1, 128, 64), (3, 5, 33), (16, 16, 16), (17, 130, 257), (64, 300, 128),
      (129, 255, 1000), (1, 4096, 4096), (8, 1000, 4099), (33, 777, 515), (100, 2048, 1024),
      (256, 256, 256), (300, 520, 384), (515, 1024, 129), (1030, 770, 640),
      (2, 777, 515), (2, 5, 33), (1, 200, 131), (4, 1000, 2049), (40, 260, 2500),
      (130, 40, 900), (2050, 20, 130), (1800, 2000, 200), (2100, 1700, 1111), (129, 12900, 64),
      (12900, 130, 384)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", MM)
def test_matmul(m, n, k, dtype):
    for pitch in (True, False):
        a, b = _ints((m, k), 1), _ints((n, k), 2)
        if pitch:
            pa, pb = ouo.int8_empty(m, k), ouo.int8_empty(n, k)
            a, b = pa.copy_(a), pb.copy_(b)
        sa = torch.rand(m, generator=_rng(3), device=DEV) + 0.1
        sb = torch.rand(n, generator=_rng(4), device=DEV) - 0.5
        # D on 16-byte boundaries (padded), or on none
        for pad, off in ((-n % 8 + 8, 0), (5, 1)):
            d = Guard(m, n, dtype, pad, off)
            ouo.int8_matmul(a, sa, b, sb, d.v)
            _check_mm(d.v, a, sa, b, sb)
            d.check()


def test_matmul_padding_is_not_read_as_data():
    """What stands between a row's end and the next row does not count."""
    a, b = ouo.int8_empty(40, 33), ouo.int8_empty(50, 33)
    for t in (a, b):
        t._base.fill_(127)
        t.copy_(_ints(t.shape, 5))
    d = torch.empty((40, 50), device=DEV)
    one = torch.ones(64, device=DEV)
    ouo.int8_matmul(a, one, b, one, d)
    _check_mm(d, a, one[:40], b, one[:50])


def test_matmul_largest_sums():
    """-128 * -128 at the deepest K: 2^14 * 131071 < 2^31, exact in 32 bits."""
    for m in (1, 200):
        k = 131071
        a, b = ouo.int8_empty(m, k).fill_(-128), ouo.int8_empty(130, k).fill_(-128)
        b[1::2].fill_(127)
        d = torch.empty((m, 130), device=DEV)
        one = torch.ones(256, device=DEV)
        ouo.int8_matmul(a, one, b, one, d)
        e = torch.tensor([16384.0 * k, -128.0 * 127 * k], dtype=torch.float64)
        # the one rounding of the integer to fp32
        assert torch.equal(d[0, :2].cpu(), e.float())
        assert (d[:, 0::2] == d[0, 0]).all() and (d[:, 1::2] == d[0, 1]).all()


def test_matmul_empty_and_nan():
    one = torch.ones(8, device=DEV)
    d = torch.full((3, 4), 77.0, device=DEV)
    ouo.int8_matmul(ouo.int8_empty(3, 0), one, ouo.int8_empty(4, 0), one, d)
    assert (d == 0).all()
    ouo.int8_matmul(ouo.int8_empty(0, 8), one, ouo.int8_empty(4, 8), one,
                    torch.empty((0, 4), device=DEV))
    ouo.int8_matmul(ouo.int8_empty(4, 8), one, ouo.int8_empty(0, 8), one,
                    torch.empty((4, 0), device=DEV))
    s = one.clone()
    s[1] = float("nan")
    a = ouo.int8_empty(3, 16).fill_(1)
    a[1] = 0
    ouo.int8_matmul(a, s, ouo.int8_empty(4, 16).fill_(1), one, d)
    assert torch.isnan(d[1]).all() and (d[[0, 2]] == 16).all()


def test_matmul_batch_of_mixed_shapes():
    """One call over many products, some sharing an operand: the bits of each
    are those it has alone."""
    shapes = [(m, n, k) for m, n, k in MM] * 5
    As = [ouo.int8_empty(m, k).copy_(_ints((m, k), i)) for i, (m, _, k) in enumerate(shapes)]
    Bs = [ouo.int8_empty(n, k).copy_(_ints((n, k), 100 + i)) for i, (_, n, k) in enumerate(shapes)]
    As[3] = _ints((16, 16), 7)[:, :16]
    sa = [torch.rand(m, generator=_rng(i), device=DEV) for i, (m, _, _) in enumerate(shapes)]
    sb = [torch.rand(n, generator=_rng(i), device=DEV) for i, (_, n, _) in enumerate(shapes)]
    Ds = [torch.empty((m, n), dtype=BF, device=DEV) for m, n, _ in shapes]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ouo.int8_matmul(As, sa, Bs, sb, Ds, status=st)
    for a, x, b, y, d in zip(As, sa, Bs, sb, Ds):
        one = torch.empty_like(d)
        ouo.int8_matmul(a, x, b, y, one)
        assert torch.equal(one, d)
        _check_mm(d, a, x, b, y)
    assert st.item() == 0


# --------------------------------------------------------------- rms_norm


def _sum_tol(n):
    # terms per thread: at most n / 32 (a row is taken by a warp or more)
    return (n / 32 + 32) * U32


NORM = [(1, 1), (1, 4096), (3, 7), (33, 70), (5, 129), (200, 2048), (700, 1000), (2, 8192),
        (3, 20001), (1300, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["tight", "pitch", "odd"])
@pytest.mark.parametrize("rows,cols", NORM)
def test_rms_norm(rows, cols, layout, dtype):
    pad, off = {"tight": (0, 0), "pitch": (24, 0), "odd": (3, 1)}[layout]
    g = _rng(rows + cols)
    x = Guard(rows, cols, dtype, pad, off, torch.randn((rows, cols), generator=g, device=DEV))
    r = Guard(rows, cols, dtype, pad, off, torch.randn((rows, cols), generator=g, device=DEV))
    w = (torch.rand(cols, generator=g, device=DEV) + 0.5).to(dtype)
    eps = 1e-5
    for res in (False, True):
        h = Guard(rows, cols, dtype, pad, off) if res else None
        y, q = Guard(rows, cols, dtype, pad, off), Guard(rows, cols, torch.int8, pad, off)
        scale, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        ouo.rms_norm(x.v, w, Y=y.v, Q=q.v, scale=scale, residual=r.v if res else None,
                     H=h.v if res else None, rstd=rstd, eps=eps)
        for t in (x, r, y, q) + ((h,) if res else ()):
            t.check()
        if res:
            # one fp32 sum, one rounding to H's type
            s = (x.v.float() + r.v.float()).to(dtype)
            assert torch.equal(h.v, s)
        ye, re = ot.rms_norm(to64(h.v if res else x.v), to64(w), eps)
        tol = _sum_tol(cols) / 2 + 4 * U32  # the square root halves the sum's error
        assert np.all(np.abs(to64(rstd) - re) <= tol * re)
        tol += 3 * U32
        assert np.all(np.abs(to64(y.v) - ye) <= (tol + UOUT[dtype]) * np.abs(ye))
        qe, se = ot.quantize(ye)
        assert np.all(np.abs(to64(scale) - se) <= (tol + 2 * U32) * se)
        assert np.all(np.abs(to64(q.v) - qe) <= 0.5 + 127 * (2 * tol + 4 * U32))


def test_rms_norm_mixed_types_and_in_place():
    """fp32 residual stream, bf16 layer, fp32 weight; H is the residual itself."""
    g = _rng(9)
    x = torch.randn((70, 1032), generator=g, device=DEV).to(BF)
    r = torch.randn((70, 1032), generator=g, device=DEV)
    w = torch.rand(1032, generator=g, device=DEV) + 0.5
    want = x.float() + r
    y = torch.empty_like(x)
    ouo.rms_norm(x, w, Y=y, residual=r, H=r, eps=0.0)
    assert torch.equal(r, want)
    ye, _ = ot.rms_norm(to64(want), to64(w), 0.0)
    assert np.all(np.abs(to64(y) - ye) <= (UOUT[BF] + _sum_tol(1032)) * np.abs(ye))
    # without a residual H takes X in its own type
    h = torch.empty_like(r)
    ouo.rms_norm(x, w, Y=y, H=h, eps=0.0)
    assert torch.equal(h, x.float())


@pytest.mark.parametrize("rows,cols", [(3, 16), (700, 1000), (1300, 2048), (333, 4096), (40, 8192),
                                       (50, 1001), (3, 20008)])
@pytest.mark.parametrize("types", [(BF, F32, BF), (BF, F32, F32), (BF, BF, F32), (F32, F32, BF),
                                   (F32, BF, F32)])
def test_rms_norm_types(rows, cols, types):
    """x / y, residual / h / gradient stream and weight of different types,
    forward and backward."""
    dt, ht, wt = types
    g = _rng(cols)
    x = torch.randn((rows, cols), generator=g, device=DEV).to(dt)
    r = torch.randn((rows, cols), generator=g, device=DEV).to(ht)
    w = (torch.rand(cols, generator=g, device=DEV) + 0.5).to(wt)
    h, y, q = torch.empty_like(r), torch.empty_like(x), ouo.int8_empty(rows, cols)
    scale, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ouo.rms_norm(x, w, Y=y, Q=q, scale=scale, residual=r, H=h, rstd=rstd, eps=1e-5)
    assert torch.equal(h, (x.float() + r.float()).to(ht))
    ye, re = ot.rms_norm(to64(h), to64(w), 1e-5)
    tol = _sum_tol(cols) / 2 + 7 * U32
    assert np.all(np.abs(to64(rstd) - re) <= tol * re)
    assert np.all(np.abs(to64(y) - ye) <= (tol + UOUT[dt]) * np.abs(ye))
    assert np.all(np.abs(to64(q) - ot.quantize(ye)[0]) <= 0.5 + 127 * (2 * tol + 4 * U32))
    dy = torch.randn((rows, cols), generator=g, device=DEV).to(dt)
    dh = torch.randn((rows, cols), generator=g, device=DEV).to(ht)
    dx, dw = torch.empty_like(dh), torch.empty(cols, device=DEV)
    ouo.rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, dH=dh)
    G, H, W, R, D = to64(dy), to64(h), to64(w), to64(rstd)[:, None], to64(dh)
    ex, ew = ot.rms_norm_grad(G, H, W, R[:, 0], D)
    mag = R * (np.abs(G * W) + np.abs(H) * R * R * np.mean(np.abs(G * W * H), 1, keepdims=True)) + np.abs(D)
    assert np.all(np.abs(to64(dx) - ex) <= (_sum_tol(cols) + 8 * U32) * mag + UOUT[ht] * np.abs(ex))
    assert np.all(np.abs(to64(dw) - ew) <= (rows + 34) * U32 * np.sum(np.abs(G * H * R), axis=0))


def test_rms_norm_zero_and_nonfinite_rows():
    x = torch.randn((5, 256), generator=_rng(1), device=DEV)
    x[1] = 0
    x[2, 5], x[3, 7] = float("nan"), float("inf")
    w = torch.ones(256, device=DEV)
    y, q, s = torch.empty_like(x), ouo.int8_empty(5, 256), torch.empty(5, device=DEV)
    ouo.rms_norm(x, w, Y=y, Q=q, scale=s, eps=1e-6)
    assert (y[1] == 0).all() and s[1] == 0 and not q[1].any()
    for i in (2, 3):
        assert torch.isnan(s[i]) and not q[i].any() and torch.isnan(y[i]).any()
    assert torch.isfinite(y[[0, 4]]).all()


def test_rms_norm_no_rows():
    e = torch.empty((0, 64), device=DEV)
    w, dw = torch.ones(64, device=DEV), torch.full((64,), 77.0, device=DEV)
    ouo.rms_norm(e, w, Y=e.clone(), rstd=torch.empty(0, device=DEV))
    ouo.rms_norm_backward(e, e, w, torch.empty(0, device=DEV), e.clone(), dweight=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["tight", "pitch", "odd"])
@pytest.mark.parametrize("rows,cols", NORM + [(5000, 72)])
def test_rms_norm_backward(rows, cols, layout, dtype):
    pad, off = {"tight": (0, 0), "pitch": (24, 0), "odd": (3, 1)}[layout]
    g = _rng(rows * 3 + cols)
    dy, h, dh = (Guard(rows, cols, dtype, pad, off,
                       torch.randn((rows, cols), generator=g, device=DEV)) for _ in range(3))
    w = (torch.rand(cols, generator=g, device=DEV) + 0.5).to(dtype)
    rstd = torch.rsqrt(h.v.float().square().mean(1) + 1e-6)
    for with_dh, with_dw in ((True, True), (False, True), (True, False)):
        dx = Guard(rows, cols, dtype, pad, off)
        dw = torch.full((cols + 1,), 77.0, device=DEV) if with_dw else None
        ouo.rms_norm_backward(dy.v, h.v, w, rstd, dx.v, dweight=dw, dH=dh.v if with_dh else None)
        dx.check()
        G, H, W, R = to64(dy.v), to64(h.v), to64(w), to64(rstd)[:, None]
        D = to64(dh.v) if with_dh else None
        ex, ew = ot.rms_norm_grad(G, H, W, R[:, 0], D)
        # magnitudes of the terms that are added
        mag = R * (np.abs(G * W) + np.abs(H) * R * R * np.mean(np.abs(G * W * H), 1, keepdims=True))
        mag = mag + (np.abs(D) if with_dh else 0)
        assert np.all(np.abs(to64(dx.v) - ex) <= (_sum_tol(cols) + 8 * U32) * mag
                      + UOUT[dtype] * np.abs(ex))
        if with_dw:
            assert dw[-1] == 77
            # every row in one run at worst, two roundings a term
            tol = (rows + 32 + 2) * U32 * np.sum(np.abs(G * H * R), axis=0)
            assert np.all(np.abs(to64(dw[:-1]) - ew) <= tol)


@pytest.mark.parametrize("into", ["dY", "dH"])
def test_rms_norm_backward_in_place_is_the_same(into):
    g = _rng(4)
    dy, h, dh = (torch.randn((333, 520), generator=g, device=DEV).to(BF) for _ in range(3))
    w, rstd = torch.rand(520, generator=g, device=DEV), torch.rand(333, generator=g, device=DEV)
    dx, dw, dw2 = torch.empty_like(dy), torch.empty(520, device=DEV), torch.empty(520, device=DEV)
    ouo.rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, dH=dh)
    out = dy if into == "dY" else dh
    ouo.rms_norm_backward(dy, h, w, rstd, out, dweight=dw2, dH=dh)
    assert torch.equal(out, dx) and torch.equal(dw, dw2)


# ----------------------------------------------------------- distillation


def _teacher(rows, vocab, k, seed, dtype=F32):
    g = _rng(seed)
    idx = torch.randint(0, vocab, (rows, k), generator=g, device=DEV)  # some twice
    t = (torch.randn((rows, k), generator=g, device=DEV) * 2 + 5).to(dtype)
    if rows > 2:
        idx[1] = -1                       # a row without entries
        idx[2, k // 2:] = vocab           # past the vocabulary: does not count
        t[0, k // 2:] = -float("inf") if k > 1 else 0.0
    return t, idx.to(torch.int32)


def _check_loss(s, t, idx, tau, loss, lse):
    le, ze = ot.distill_loss(to64(s), to64(t), idx.cpu().numpy(), tau)
    # s / tau is s * fl(1 / tau): 2 roundings; the exponent's error is that of
    # numbers up to z (2 roundings more) and of the exponential (2 ulp); the
    # sum's runs are at most V / 128 long, rescaled at most as often
    z = max(1.0, float(np.abs(to64(s)[np.isfinite(to64(s)) & (np.abs(to64(s)) < 1e30)]).max()) / tau)
    tt = to64(t)[np.isfinite(to64(t))]
    zt = float(np.abs(tt).max()) / tau if tt.size else 1.0
    rel = (2 * s.shape[1] / 128 + 64 + 8 * z) * U32
    assert np.all(np.abs(to64(lse) - ze) <= rel + 4 * U32 * z)
    fin = np.isfinite(le)
    assert np.array_equal(fin, np.isfinite(to64(loss)))
    err = np.abs(to64(loss)[fin] - le[fin])
    # p's error (K terms, exponents up to zt) times the spread of its factors
    prel = (t.shape[1] + 32 + 8 * zt) * U32
    assert np.all(err <= tau * tau * (rel + 4 * U32 * z + prel * (4 * z + 2 * zt + 24)))


KD = [(1, 1, 1), (1, 50001, 20), (3, 7, 3), (5, 1000, 1), (33, 4099, 64), (70, 2048, 7),
      (2, 131072, 128), (9, 32768, 1024), (300, 515, 33), (700, 64, 5)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("rows,vocab,k", KD)
def test_distill(rows, vocab, k, tau, dtype):
    for pad, off in ((0, 0), (8, 0), (3, 1)):
        s = Guard(rows, vocab, dtype, pad, off,
                  torch.randn((rows, vocab), generator=_rng(vocab), device=DEV) * 3)
        t, idx = _teacher(rows, vocab, k, 5, dtype)
        loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        ouo.distill_loss(s.v, t, idx, loss, lse, temperature=tau)
        _check_loss(s.v, t, idx, tau, loss, lse)
        s.check()
        dl = torch.randn(rows, generator=_rng(6), device=DEV)
        ds = Guard(rows, vocab, dtype, pad, off)
        ouo.distill_loss_backward(s.v, t, idx, lse, dl, ds.v, temperature=tau)
        ds.check()
        e = ot.distill_grad(to64(s.v), to64(t), idx.cpu().numpy(), to64(lse), to64(dl), tau)
        z = float(s.v.float().abs().max()) / tau + float(lse.abs().max())
        zt = float(to64(t)[np.isfinite(to64(t))].max()) / tau
        q = np.abs(e) + (np.abs(to64(dl)) * tau)[:, None] * 2  # no term is above 1
        tol = (8 * z + 8 * zt + k + 64) * U32 * np.minimum(q, 2 * (np.abs(to64(dl)) * tau)[:, None] + 1)
        assert np.all(np.abs(to64(ds.v) - e) <= tol + UOUT[dtype] * np.abs(e))
        # the same on top of the logits
        ouo.distill_loss_backward(s.v, t, idx, lse, dl, s.v, temperature=tau)
        assert torch.equal(s.v, ds.v)


def test_distill_gradient_of_small_probabilities():
    """Away from the teacher's entries the gradient is dloss tau q, to a few
    roundings of each value, however small."""
    s = torch.randn((4, 3001), generator=_rng(0), device=DEV) * 8
    t, idx = _teacher(4, 3001, 6, 1)
    idx[1] = 0
    loss, lse, dl = (torch.ones(4, device=DEV) for _ in range(3))
    ouo.distill_loss(s, t, idx, loss, lse)
    ds = torch.empty_like(s)
    ouo.distill_loss_backward(s, t, idx, lse, dl, ds)
    e = np.exp(to64(s) - to64(lse)[:, None])
    away = np.ones_like(e, dtype=bool)
    np.put_along_axis(away, np.clip(idx.cpu().numpy().astype(np.int64), 0, 3000), False, axis=1)
    # exponents up to 80: 80 * 3 roundings, and the exponential's own 2 ulp;
    # what is below 2^-126 may be flushed to zero
    tol = (80 * 3 + 8) * U32 * e + 2.0 ** -126
    assert np.all(np.abs(to64(ds) - e)[away] <= tol[away])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_distill_masked_logits(dtype):
    s = (torch.randn((4, 777), generator=_rng(2), device=DEV)).to(dtype)
    t, idx = _teacher(4, 777, 8, 3)
    idx[:, :] = torch.arange(8, device=DEV, dtype=torch.int32) * 3
    t[:] = torch.randn((4, 8), generator=_rng(4), device=DEV)
    s[0, 100:] = -float("inf")
    s[1, 100:] = torch.finfo(dtype).min
    s[2, 3] = -float("inf")  # where the teacher has weight: infinite loss
    s[3, 0] = -float("inf")  # where the teacher has none
    t[3, 0] = -float("inf")
    loss, lse = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse)
    assert torch.isinf(loss[2]) and loss[2] > 0
    _check_loss(s, t, idx, 1.0, loss, lse)
    ds = torch.empty((4, 777), device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, torch.ones(4, device=DEV), ds)
    e = ot.distill_grad(to64(s), to64(t), idx.cpu().numpy(), to64(lse), np.ones(4), 1.0)
    assert np.abs(to64(ds) - e).max() <= 200 * U32
    assert (ds[:2, 100:] == 0).all()


def test_distill_teacher_of_lowest_values():
    """A teacher row whose entries are all the type's lowest value is uniform."""
    s = torch.randn((2, 50), generator=_rng(2), device=DEV)
    t = torch.full((2, 4), torch.finfo(F32).min, device=DEV)
    t[1, 0] = 1.0
    idx = torch.tensor([[1, 2, 3, 4]] * 2, device=DEV, dtype=torch.int32)
    loss, lse = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse)
    e = ot.distill_loss(to64(s), np.array([[0.0] * 4, [1.0] + [-1e30] * 3]), idx.cpu().numpy(), 1.0)
    assert np.abs(to64(loss) - e[0]).max() <= 200 * U32


def test_distill_skipped_rows_may_hold_anything():
    s = torch.randn((4, 333), generator=_rng(2), device=DEV)
    t, idx = _teacher(4, 333, 5, 3)
    s[1] = float("nan")  # has no entries
    s[3] = float("nan")  # has dloss 0
    t[3] = float("nan")
    loss, lse = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse)
    assert loss[1] == 0 and lse[1] == 0 and torch.isnan(loss[3]) and torch.isnan(lse[3])
    dl = torch.ones(4, device=DEV)
    dl[3] = 0
    ds = torch.full((4, 333), 77.0, device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, dl, ds)
    assert (ds[1] == 0).all() and (ds[3] == 0).all() and torch.isfinite(ds).all()
    s[0, 5] = float("nan")
    ouo.distill_loss(s, t, idx, loss, lse)
    assert torch.isnan(loss[0]) and torch.isfinite(loss[2])


def test_distill_no_rows():
    e = torch.empty((0, 10), device=DEV)
    i = torch.empty((0, 3), device=DEV, dtype=torch.int32)
    z = torch.empty(0, device=DEV)
    ouo.distill_loss(e, torch.empty((0, 3), device=DEV), i, z, z)
    ouo.distill_loss_backward(e, torch.empty((0, 3), device=DEV), i, z, z, e)


# ------------------------------------------------------ past 2^31 elements


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements (and bytes): the last rows are
    those of the same rows alone."""
    last, tail = 3, lambda t: t[-3:].clone()
    rows, vocab = 16500, 131072
    s = torch.empty((rows, vocab), dtype=BF, device=DEV)
    s[-last:] = torch.randn((last, vocab), generator=_rng(0), device=DEV) * 2
    s[:-last] = 1.0
    t, idx = _teacher(rows, vocab, 4, 1)
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse)
    a, b = torch.empty(last, device=DEV), torch.empty(last, device=DEV)
    keep = tail(s)
    ouo.distill_loss(keep, tail(t), tail(idx), a, b)
    # the sums' order may be another with so few rows
    assert torch.allclose(lse[-last:], b, rtol=4 * U32, atol=0)
    assert torch.allclose(loss[-last:], a, rtol=1e-5, atol=1e-5)
    dl = torch.ones(rows, device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, dl, s)
    d = torch.empty_like(keep)
    ouo.distill_loss_backward(keep, tail(t), tail(idx), lse[-last:].contiguous(), dl[:last], d)
    assert torch.equal(s[-last:], d)
    # s again: 131072 columns as rows of 8-bit integers, both ways
    x = s.view(rows * 16, vocab // 16)
    x[-last:] = torch.randn((last, vocab // 16), generator=_rng(2), device=DEV)
    q, sc = ouo.int8_empty(*x.shape), torch.empty(x.shape[0], device=DEV)
    ouo.quantize_int8(x, q, sc)
    _check_quant(to64(q[-last:]), to64(sc[-last:]), to64(x[-last:]))
    ouo.rms_norm(x, torch.ones(x.shape[1], device=DEV), Q=q, scale=sc, eps=0.0)
    y = ot.rms_norm(to64(x[-last:]), np.ones(x.shape[1]), 0.0)[0]
    assert np.all(np.abs(to64(q[-last:]) - ot.quantize(y)[0]) <= 0.5 + 127 * _sum_tol(8192) * 2)
    qt, st = ouo.int8_empty(x.shape[1], x.shape[0]), torch.empty(x.shape[1], device=DEV)
    ouo.quantize_int8(x, qt, st, transpose=True)
    cols = x[:, -last:].t().contiguous()
    _check_quant(to64(qt[-last:]), to64(st[-last:]), to64(cols))
    del s, x, q, qt
    a8, b8 = ouo.int8_empty(66000, 64).copy_(_ints((66000, 64), 3)), ouo.int8_empty(33000, 64).copy_(_ints((33000, 64), 4))
    sa, sb = torch.rand(66000, device=DEV), torch.rand(33000, device=DEV)
    D = torch.empty((66000, 33000), dtype=BF, device=DEV)
    ouo.int8_matmul(a8, sa, b8, sb, D)
    _check_mm(D[-last:], a8[-last:], sa[-last:], b8, sb)


# ------------------------------------------------- streams, graphs, repeats


def _all_calls(seed, tokens=130, dim=520, vocab=1000):
    """Inputs and a function that runs every operator once; its outputs."""
    g = _rng(seed)
    x = torch.randn((tokens, dim), generator=g, device=DEV).to(BF)
    r = torch.randn((tokens, dim), generator=g, device=DEV).to(BF)
    w = torch.rand(dim, generator=g, device=DEV).to(BF)
    W = torch.randn((vocab, dim), generator=g, device=DEV).to(BF)
    t, idx = _teacher(tokens, vocab, 16, seed)
    dl = torch.full((tokens,), 1.0 / tokens, device=DEV)
    e = lambda *s, d=F32: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    o = dict(h=e(tokens, dim, d=BF), q=ouo.int8_empty(tokens, dim), qs=e(tokens), rstd=e(tokens),
             wq=ouo.int8_empty(vocab, dim), ws=e(vocab), wtq=ouo.int8_empty(dim, vocab), wts=e(dim),
             s=e(tokens, vocab, d=BF), loss=e(tokens), lse=e(tokens), ds=e(tokens, vocab, d=BF),
             dq=ouo.int8_empty(tokens, vocab), dqs=e(tokens), dtq=ouo.int8_empty(vocab, tokens),
             dts=e(vocab), y=e(tokens, dim, d=BF), ytq=ouo.int8_empty(dim, tokens), yts=e(dim),
             dy=e(tokens, dim, d=BF), dW=e(vocab, dim), dx=e(tokens, dim, d=BF), dw=e(dim))

    def run(**kw):
        ouo.rms_norm(x, w, Y=o["y"], Q=o["q"], scale=o["qs"], residual=r, H=o["h"], rstd=o["rstd"],
                     **kw)
        ouo.quantize_int8(W, o["wq"], o["ws"], **kw)
        ouo.quantize_int8(W, o["wtq"], o["wts"], transpose=True, **kw)
        ouo.int8_matmul(o["q"], o["qs"], o["wq"], o["ws"], o["s"], **kw)
        ouo.distill_loss(o["s"], t, idx, o["loss"], o["lse"], **kw)
        ouo.distill_loss_backward(o["s"], t, idx, o["lse"], dl, o["ds"], **kw)
        ouo.quantize_int8(o["ds"], o["dq"], o["dqs"], **kw)
        ouo.quantize_int8(o["ds"], o["dtq"], o["dts"], transpose=True, **kw)
        ouo.quantize_int8(o["y"], o["ytq"], o["yts"], transpose=True, **kw)
        ouo.int8_matmul(o["dq"], o["dqs"], o["wtq"], o["wts"], o["dy"], **kw)
        ouo.int8_matmul(o["dtq"], o["dts"], o["ytq"], o["yts"], o["dW"], **kw)
        ouo.rms_norm_backward(o["dy"], o["h"], w, o["rstd"], o["dx"], dweight=o["dw"], **kw)

    return (x, r, w, W, t, idx, dl), o, run


def test_another_stream_and_repeats_are_bit_identical():
    _, o, run = _all_calls(0)
    run()
    torch.cuda.synchronize()
    first = {k: v.clone() for k, v in o.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for v in o.values():
        v.zero_()
    s.wait_stream(torch.cuda.current_stream())
    run(stream=s)
    s.synchronize()
    for k in o:
        assert torch.equal(o[k], first[k]), k


def test_two_graphs_replayed_in_turn():
    sets = [_all_calls(seed) for seed in (1, 2)]
    want = []
    for _, o, run in sets:
        run()
        want.append({k: v.clone() for k, v in o.items()})
    graphs = []
    for _, o, run in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for _, o, _ in sets:
        for v in o.values():
            v.zero_()
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for (_, o, _), w in zip(sets, want):
        for k in o:
            assert torch.equal(o[k], w[k]), k


def test_training_step_into_the_optimizer():
    """Norm, 8-bit head, distillation, gradients, and the weight gradient
    through momentum, selection, Gram Newton-Schulz, the update and the
    weight's 8-bit copy again; each stage against the oracle on the stage's
    own inputs, the gradient within what 8 bits allow."""
    (x, r, w, W, t, idx, dl), o, run = _all_calls(3)
    run()
    H = to64(o["h"])
    y, rstd = ot.rms_norm(H, to64(w), 1e-6)
    S = ot.int8_matmul(o["q"].cpu().numpy(), to64(o["qs"]), o["wq"].cpu().numpy(), to64(o["ws"]))
    assert np.all(np.abs(to64(o["s"]) - S) <= (UOUT[BF] + 4 * U32) * np.abs(S))
    _check_loss(o["s"], t, idx, 1.0, o["loss"], o["lse"])
    dS, X = to64(o["ds"]), to64(o["y"])
    # 8-bit operands: half a step of each, summed over the tokens
    a, b = np.abs(dS).max(0) / 254, np.abs(X).max(0) / 254
    slack = (np.abs(dS).sum(0)[:, None] * b + a[:, None] * np.abs(X).sum(0)
             + dS.shape[0] * a[:, None] * b)
    assert np.all(np.abs(to64(o["dW"]) - dS.T @ X) <= slack * 1.001 + 1e-12)
    dx, dw = ot.rms_norm_grad(to64(o["dy"]), H, to64(w), to64(o["rstd"]))
    assert np.abs(to64(o["dw"]) - dw).max() <= 200 * U32 * np.abs(to64(o["dy"]) * H * rstd[:, None]).sum(0).max()

    M, before = torch.zeros_like(o["dW"]), W.clone()
    keys = torch.empty(M.shape[0], dtype=torch.float64, device=DEV)
    ouo.dion_momentum_update([M], [o["dW"]], 0.95, "accum", keys)
    assert torch.equal(M, o["dW"])
    k = ouo.dion3_num_selected(M.shape[0], 0.125)
    sel = torch.empty(k, dtype=torch.int32, device=DEV)
    X0, sc = ouo.batch_empty([(k, M.shape[1])], BF, DEV), torch.empty(1, device=DEV)
    ouo.dion3_select_rows([M], keys, 0.125, sel, X0, sc)
    O = [torch.empty_like(X0[0])]
    ouo.gram_ns_orthogonalize(X0, O, ouo.ns_params(normalize=False))
    ouo.apply_update([W], O, lr=0.5, idx=sel)
    ouo.quantize_int8(W, o["wq"], o["ws"])
    moved = torch.zeros(W.shape[0], dtype=torch.bool, device=DEV)
    moved[sel.long()] = True
    assert torch.equal(W[~moved], before[~moved]) and not torch.equal(W[moved], before[moved])
    _check_quant(o["wq"].cpu().numpy().astype(np.float64), to64(o["ws"]), to64(W))
    loss = o["loss"].sum().item()
    run()
    assert np.isfinite(loss) and torch.isfinite(o["loss"]).all()
