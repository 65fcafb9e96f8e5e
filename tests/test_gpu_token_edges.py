"""GPU tests of the token-matrix operators where they are easiest to get
wrong."""
import numpy as np
import pytest
import torch

import orthonormalized_update_optimizers_b200 as ouo
from oracle import tokens as ot
from orthonormalized_update_optimizers_b200._lib import OuoError

from ._util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
U32 = 2.0 ** -24  # half a step of fp32


# ------------------------------------------------------ ties of the rounding


def _even(num, den):
    """num / den rounded to nearest, ties to even, in integers (num >= 0)."""
    q = num // den
    r = 2 * (num - q * den)
    return np.where(r > den, q + 1, np.where(r < den, q, q + (q & 1)))


def _bf16_rows():
    """A row for each of bf16's 128 mantissas as the largest magnitude, with
    every bf16 value down to 2^-9 of it, both signs: (x, exact q)."""
    e = np.repeat(np.arange(10), 128)
    m = np.tile(np.arange(128, 256), 10)
    xs, qs = [], []
    for a in range(128, 256):
        keep = m <= a << e  # at most the largest
        x, q = m / 2.0 ** e * keep, _even(127 * m * keep, a << e)
        xs.append(np.concatenate([[a], x, -x]))
        qs.append(np.concatenate([[127], q, -q]))
    return np.array(xs), np.array(qs)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("copies", [1, 20])  # 20: past the 3 MB of the one-read transposition
@pytest.mark.parametrize("pad", [7, 8])      # element by element, and in 16 bytes
def test_quantize_rounds_every_bf16_value_exactly(dtype, transpose, copies, pad):
    x, q = _bf16_rows()
    x, q = np.tile(x, (copies, 1)), np.tile(q, (copies, 1))
    m, n = x.shape
    x = np.concatenate([x, np.zeros((m, pad))], 1)
    q = np.concatenate([q, np.zeros((m, pad))], 1)
    t = torch.tensor(x, device=DEV).to(dtype)
    assert np.array_equal(to64(t), x)
    if transpose:
        t = t.t().contiguous()
    got, scale = ouo.int8_empty(m, n + pad), torch.empty(m, device=DEV)
    ouo.quantize_int8(t, got, scale, transpose=transpose)
    assert np.array_equal(to64(got), q)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("power", [0, -110, 40])
def test_quantize_ties_of_fp32_rows(transpose, power):
    """Rows whose scale is b 2^power: x = (k + 1/2) b 2^power is a tie."""
    k = np.arange(-127, 127)
    even = np.where(k % 2 == 0, k, k + 1)
    b = np.array([1, 3, 5, 7, 9, 127, 1001, 32767, 65535])[:, None]
    x = np.concatenate([127.0 * b, (k + 0.5) * b], 1) * 2.0 ** power
    t = torch.tensor(x, dtype=F32, device=DEV)
    assert np.array_equal(to64(t), x)
    got, scale = ouo.int8_empty(*x.shape), torch.empty(len(b), device=DEV)
    ouo.quantize_int8(t.t().contiguous() if transpose else t, got, scale, transpose=transpose)
    assert np.array_equal(to64(scale), b[:, 0] * 2.0 ** power)
    assert np.array_equal(to64(got)[:, 1:], np.tile(even, (len(b), 1))) and (got[:, 0] == 127).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [2560, 2561, 20480])
def test_rms_norm_rounds_ties_to_even(cols, dtype):
    """h = +-1 and eps = 0 make the norm's output +-weight, exactly."""
    x, q = _bf16_rows()
    h = torch.ones((2, cols), dtype=dtype, device=DEV)
    h[1, ::2] = -1
    sign = to64(h)
    got, scale = ouo.int8_empty(2, cols), torch.empty(2, device=DEV)
    for a in range(0, 128, 9):
        w = torch.tensor(np.resize(x[a], cols), device=DEV).to(dtype)
        ouo.rms_norm(h, w, Q=got, scale=scale, eps=0.0)
        assert np.array_equal(to64(got), sign * np.resize(q[a], cols))


# ------------------------------------------------------ outputs over inputs


def test_outputs_over_inputs_are_refused():
    """By the host, before a launch: every buffer is as it was."""
    x = torch.randn((40, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    r, h, y = torch.randn_like(x), torch.empty_like(x), torch.empty_like(x)
    v = torch.empty(40, device=DEV)
    i8 = x.view(torch.int8)  # 40 x 256
    q = ouo.int8_empty(40, 64)
    t, idx = torch.randn((40, 4), device=DEV), torch.zeros((40, 4), dtype=torch.int32, device=DEV)
    a, b = torch.zeros((40, 64), dtype=torch.int8, device=DEV), ouo.int8_empty(16, 64).zero_()
    wide = torch.randn((40, 128), device=DEV)
    keep = [k.clone() for k in (x, w, r, t, a, wide)]
    rms, bwd, kd, kdb = ouo.rms_norm, ouo.rms_norm_backward, ouo.distill_loss, ouo.distill_loss_backward
    calls = [
        ("Q and X", lambda: ouo.quantize_int8(x, i8[:, :64], v)),
        ("scale and X", lambda: ouo.quantize_int8(x, q, x[0])),
        ("D and A", lambda: ouo.int8_matmul(a, v, b, w, a.view(torch.float32)[:, :16])),
        ("D and b_scale", lambda: ouo.int8_matmul(a[:1], v, b, w, w[None, 8:24])),
        ("Y and X", lambda: rms(x, w, Y=x, Q=q, scale=v)),
        ("Y and residual", lambda: rms(x, w, Y=r, residual=r, H=h)),
        ("H and Y", lambda: rms(x, w, Y=r, residual=r, H=r)),
        ("H and X", lambda: rms(x[1:], w, Y=y[1:], H=x[:39])),
        ("Q and X", lambda: rms(x, w, Q=i8[:, :64], scale=v)),
        ("rstd and weight", lambda: rms(x, w, Y=y, rstd=w)),
        ("scale and rstd", lambda: rms(x, w, Q=q, scale=v, rstd=v)),
        ("Y and X", lambda: rms(wide[:, :64], w, Y=wide[:, 32:96])),
        ("dX and H", lambda: bwd(x, r, w, v, r)),
        ("dX and dY", lambda: bwd(x[1:], r[1:], w, v, x[:39])),
        ("dX and dH", lambda: bwd(y[1:], r[1:], w, v, x[:39], dH=x[1:])),
        ("dweight and weight", lambda: bwd(x, r, w, v, y, dweight=w)),
        ("dX and dweight", lambda: bwd(x, r, w, v, y, dweight=y[1])),
        ("loss and S", lambda: kd(x, t, idx, x[0], v)),
        ("loss and lse", lambda: kd(x, t, idx, v, v)),
        ("dS and S", lambda: kdb(x[1:], t[1:], idx[1:], v, v, x[:39])),
        ("dS and teacher", lambda: kdb(x[:, :4], t, idx, v, v, t)),
    ]
    for what, call in calls:
        with pytest.raises(OuoError, match=what + " overlap"):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(k, m) for k, m in zip(keep, (x, w, r, t, a, wide)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [64, 1000, 4097, 20001])
def test_rms_norm_in_place(cols, dtype):
    x = torch.randn((9, cols), device=DEV).to(dtype)
    w = torch.rand(cols, device=DEV).to(dtype)
    y, r1, r2 = torch.empty_like(x), torch.empty(9, device=DEV), torch.empty(9, device=DEV)
    ouo.rms_norm(x, w, Y=y, rstd=r1)
    ouo.rms_norm(x, w, Y=x, rstd=r2)
    assert torch.equal(x, y) and torch.equal(r1, r2)


def test_columns_of_one_buffer():
    """Inputs and outputs that are columns of one wider matrix are apart."""
    buf = torch.randn((33, 3 * 128), device=DEV)
    x, y, h = buf[:, :128], buf[:, 128:256], buf[:, 256:]
    w, keep = torch.rand(128, device=DEV), x.clone()
    want = torch.empty_like(keep)
    ouo.rms_norm(keep, w, Y=want)
    ouo.rms_norm(x, w, Y=y, H=h)
    assert torch.equal(x, keep) and torch.equal(y, want) and torch.equal(h, keep)


# ------------------------------------------------------ workspaces and streams


def test_workspace_of_another_stream_is_not_one_that_is_still_in_use():
    """The current stream keeps writing to a buffer that the host has given
    back; calls on another stream that take a workspace of that size."""
    rows, cols = 4096, 2048
    x = torch.randn((rows, cols), device=DEV).to(BF)
    w, rstd = torch.ones(cols, device=DEV), torch.ones(rows, device=DEV)
    q, sc = ouo.int8_empty(cols, rows), torch.empty(cols, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)

    def run(**kw):
        ouo.quantize_int8(x, q, sc, transpose=True, **kw)
        ouo.rms_norm_backward(x, x, w, rstd, dx, dweight=dw, **kw)

    run()
    want = [t.clone() for t in (q, sc, dx, dw)]
    sizes = (ouo.quantize_int8_workspace_bytes(x, True),
             ouo.rms_norm_backward_workspace_bytes(rows, cols))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        held = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]
        for _ in range(200):
            for t in held:
                t.fill_(255)
        del held, t
        run(stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, sc, dx, dw), want))
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_batch_of_all_kinds(dtype):
    """Aligned, odd, long and empty matrices in one call: each as alone, and
    each kind in a launch of its own."""
    g = torch.Generator(DEV).manual_seed(1)
    shapes = [(70, 256), (3, 20000), (9, 129), (0, 7), (4, 0), (300, 1024), (2, 16385), (5, 16384),
              (1, 1), (33, 8)]
    xs = [torch.randn(s, generator=g, device=DEV).to(dtype) for s in shapes]
    xs.append(torch.randn((8, 65), generator=g, device=DEV).to(dtype)[:, 1:])  # odd pitch, 64 wide
    qs = [ouo.int8_empty(*x.shape).fill_(7) for x in xs]
    ss = [torch.full((x.shape[0] + 1,), 77.0, device=DEV) for x in xs]

    def launches(*args):
        before = ouo.launch_count()
        ouo.quantize_int8(*args)
        return ouo.launch_count() - before

    assert launches(xs, qs, ss) == 3
    for x, q, s in zip(xs, qs, ss):
        one, so = ouo.int8_empty(*x.shape), torch.full((x.shape[0] + 1,), 77.0, device=DEV)
        assert launches(x, one, so) == (x.shape[0] > 0)
        assert torch.equal(q, one) and torch.equal(s, so)
    # an empty matrix has no say, whatever its length
    assert launches([xs[0], xs[3]], [qs[0], qs[3]], [ss[0], ss[3]]) == 1


# ------------------------------------------- temperatures far from the usual


def _near_teacher(rows, vocab, dtype, seed):
    """Logits, and a teacher that has every entry of the vocabulary, near them."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = torch.randn((rows, vocab), generator=g, device=DEV).to(dtype)
    idx = torch.stack([torch.randperm(vocab, generator=g, device=DEV) for _ in range(rows)])
    t = s.float().gather(1, idx) + 0.3 * torch.randn((rows, vocab), generator=g, device=DEV)
    return s, t, idx.to(torch.int32)


TAUS = [1e-3, 1e-2, 0.3, 1.0, 4.0, 4.5, 20.0, 100.0, 1000.0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tau", TAUS)
@pytest.mark.parametrize("vocab", [10, 1000])
def test_distill_loss_keeps_its_digits_at_any_temperature(vocab, tau, dtype):
    s, t, idx = _near_teacher(4, vocab, dtype, 3)
    loss, lse = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse, temperature=tau)
    # the operator divides by tau as a product with the fp32 number nearest to 1 / tau
    inv = float(np.float32(1) / np.float32(tau))
    le, ze = ot.distill_loss(to64(s), to64(t), idx.cpu().numpy(), 1 / inv)
    le = le * (float(np.float32(tau)) * inv) ** 2
    x = to64(s)
    d = (x.max(1, keepdims=True) - x) * inv
    Z = np.exp(-d).sum(1)
    if tau <= 4:
        # the exponential: 2 ulp, its argument three roundings; a thread's sum
        # of vocab / 128 terms, in eights, and the block's
        eps = 4 * U32 + 3 * U32 * (d * np.exp(-d)).sum(1) / Z + (vocab / 1024 + 24) * U32
        # the teacher's: as much in the sum, and in each p (all of them cover
        # the vocabulary; the logits are 0.3 apart, five times that at most)
        both = 2 * eps + (eps + 4 * U32 + 3 * U32 * d.max(1)) * 2 * 5 * 0.3 * inv
    else:
        # what is summed is within 14 roundings of e^d - 1, at most 1.8 |d|: two
        # in d, four in the series (or the exponential and the 1), four in sums of
        # eight; m may be below the logit, by d = 1 at most.  The teacher in float64.
        both = eps = 14 * U32 * np.maximum(d, np.minimum(1, d.max(1, keepdims=True))).sum(1) / Z
    assert np.all(np.abs(to64(loss) - le) <= tau * tau * both + 2 * U32 * np.abs(le))
    assert np.all(np.abs(to64(lse) - ze) <= eps + 2 * U32 * np.abs(ze))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tau", TAUS)
def test_distill_gradient_keeps_its_digits_at_any_temperature(tau, dtype):
    vocab = 1000
    s, t, idx = _near_teacher(4, vocab, dtype, 4)
    loss, lse, dl = (torch.ones(4, device=DEV) for _ in range(3))
    ouo.distill_loss(s, t, idx, loss, lse, temperature=tau)
    ds = torch.empty((4, vocab), device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, dl, ds, temperature=tau)
    inv = float(np.float32(1) / np.float32(tau))
    e = ot.distill_grad(to64(s), to64(t), idx.cpu().numpy(), to64(lse), to64(dl), 1 / inv)
    e = e * float(np.float32(tau)) * inv
    x = to64(s) * inv - to64(lse)[:, None]
    q = np.exp(x)
    T = np.empty_like(x)
    np.put_along_axis(T, idx.cpu().numpy().astype(np.int64), to64(t), 1)
    d = (T.max(1, keepdims=True) - T) * inv
    p = np.exp(-d) / np.exp(-d).sum(1, keepdims=True)
    # q: a fused product, log2(e) (2), the exponential (2 ulp); p: d (2), the
    # exponential (2), the sum of 1000 / 128 terms and the block's, 1 / z (2)
    eq = (4 * np.abs(x) + 4) * U32 * q
    ep = (2 * d + 3 * np.sum(p * d, 1, keepdims=True) + 8 + 8 + 12) * U32 * p
    # the difference and two products; tiny probabilities may be flushed
    tol = tau * (eq + ep + 2.0 ** -126) + 4 * U32 * np.abs(e)
    assert np.all(np.abs(to64(ds) - e) <= tol)


@pytest.mark.parametrize("tau", [0.25, 0.7, 1.0, 8.0])
def test_distill_teacher_of_lowest_values_at_any_temperature(tau):
    """Entries that all have the lowest value count, equally, although the
    quotient by the temperature is not finite."""
    s = torch.randn((2, 50), generator=torch.Generator(DEV).manual_seed(2), device=DEV)
    t = torch.full((2, 4), torch.finfo(F32).min, device=DEV)
    t[1, 0] = 1.0
    idx = torch.tensor([[1, 2, 3, 4]] * 2, device=DEV, dtype=torch.int32)
    loss, lse = torch.empty(2, device=DEV), torch.empty(2, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse, temperature=tau)
    near = np.array([[0.0] * 4, [1.0] + [-1e30] * 3])
    le, ze = ot.distill_loss(to64(s), near, idx.cpu().numpy(), tau)
    # the tolerance of the masked rows at temperature 1, times tau^2
    assert np.abs(to64(loss) - le).max() <= 200 * U32 * max(1.0, tau * tau)
    ds, dl = torch.empty_like(s), torch.ones(2, device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, dl, ds, temperature=tau)
    e = ot.distill_grad(to64(s), near, idx.cpu().numpy(), to64(lse), np.ones(2), tau)
    assert np.abs(to64(ds) - e).max() <= 200 * U32 * max(1.0, tau)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,vocab", [(2, 131072), (33, 4099), (700, 64), (300, 50001)])
def test_distill_high_temperature_over_shapes(rows, vocab, dtype):
    """Clusters, odd rows and short ones; masked and skipped entries."""
    tau, k = 50.0, 32
    g = torch.Generator(DEV).manual_seed(5)
    s = (torch.randn((rows, vocab), generator=g, device=DEV) * 3).to(dtype)
    s[0, 5:9] = -float("inf")
    s[1, 5:9] = torch.finfo(dtype).min
    t = torch.randn((rows, k), generator=g, device=DEV)
    idx = torch.randint(9, vocab, (rows, k), generator=g, device=DEV).to(torch.int32)
    if rows > 2:
        idx[2] = -1
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse, temperature=tau)
    inv = float(np.float32(1) / np.float32(tau))
    le, ze = ot.distill_loss(to64(s), to64(t), idx.cpu().numpy(), 1 / inv)
    le = le * (float(np.float32(tau)) * inv) ** 2
    x = to64(s)
    d = np.minimum((x.max(1, keepdims=True) - x) * inv, 1e3)
    # as above; where logits are masked, e^d - 1 is -1
    far = np.minimum(1, np.where(d < 1e3, d, 0).max(1, keepdims=True))
    eps = 14 * U32 * np.minimum(np.maximum(d, far), 2.0).sum(1) / np.exp(-d).sum(1)
    assert np.all(np.abs(to64(loss) - le) <= tau * tau * eps + 2 * U32 * np.abs(le))
    assert np.all(np.abs(to64(lse) - ze) <= eps + 2 * U32 * np.abs(ze))


# ------------------------------------------------ depths past sums of 32 bits


def _ints(shape, seed, lo=-127, hi=127):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int8)


def _exact_product(a, sa, b, sb):
    """In float64, where these sums are exact."""
    e = a.double() @ b.double().t()
    assert e.abs().max() < 2 ** 53
    return (e * sa.double()[:, None] * sb.double()).cpu().numpy()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,n,k", [
    (1, 130, 131072), (2, 70, 152064), (5, 33, 131072), (30, 260, 200001), (64, 40, 131200),
    (200, 300, 152064), (300, 100, 256000), (3, 7, 1047552), (130, 129, 131072)])
@pytest.mark.parametrize("extreme", [False, True])
def test_deep_product(m, n, k, dtype, extreme):
    if extreme:  # every sum as large as it gets, or as small
        a, b = ouo.int8_empty(m, k).fill_(-128), ouo.int8_empty(n, k).fill_(-128)
        b[1::2].fill_(127)
    else:
        a = ouo.int8_empty(m, k).copy_(_ints((m, k), 1))
        b = ouo.int8_empty(n, k).copy_(_ints((n, k), 2))
    sa = torch.rand(m, device=DEV) + 0.1
    sb = torch.rand(n, device=DEV) - 0.5
    d = torch.full((m, n + 5), 77.0, dtype=dtype, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ouo.int8_matmul(a, sa, b, sb, d[:, :n], status=st)
    e = _exact_product(a, sa, b, sb)
    tol = (1 + {BF: 2.0 ** -8, F32: U32}[dtype]) * (1 + U32) ** 3 - 1
    assert np.all(np.abs(to64(d[:, :n]) - e) <= tol * np.abs(e))
    assert (d[:, n:] == 77).all() and st.item() == 0


@pytest.mark.parametrize("m,n,k", [(1, 9, 131073), (70, 66, 131072), (5, 130, 300001)])
@pytest.mark.parametrize("extreme", [False, True])
def test_deep_product_of_unaligned_rows(m, n, k, extreme):
    def rows(r, seed):
        if extreme:
            return torch.full((r, k + 1), -128, dtype=torch.int8, device=DEV)[:, 1:]
        return _ints((r, k + 1), seed)[:, 1:]

    a, b = rows(m, 1), rows(n, 2)
    sa, sb = torch.rand(m, device=DEV), torch.rand(n, device=DEV)
    d = torch.empty((m, n), device=DEV)
    ouo.int8_matmul(a, sa, b, sb, d)
    e = _exact_product(a, sa, b, sb)
    assert np.all(np.abs(to64(d) - e) <= ((1 + U32) ** 4 - 1) * np.abs(e))


def test_deep_products_in_a_batch():
    """Beside products of ordinary depth; each as it is alone."""
    shapes = [(3, 40, 64), (3, 40, 131072), (300, 300, 256), (20, 500, 152064), (1, 16, 140000)]
    As = [ouo.int8_empty(m, k).copy_(_ints((m, k), i)) for i, (m, _, k) in enumerate(shapes)]
    Bs = [ouo.int8_empty(n, k).copy_(_ints((n, k), 9 + i)) for i, (_, n, k) in enumerate(shapes)]
    sa = [torch.rand(m, device=DEV) for m, _, _ in shapes]
    sb = [torch.rand(n, device=DEV) for _, n, _ in shapes]
    Ds = [torch.empty((m, n), device=DEV) for m, n, _ in shapes]
    ouo.int8_matmul(As, sa, Bs, sb, Ds)
    for a, x, b, y, d in zip(As, sa, Bs, sb, Ds):
        one = torch.empty_like(d)
        ouo.int8_matmul(a, x, b, y, one)
        e = _exact_product(a, x, b, y)
        assert torch.equal(one, d)
        assert np.all(np.abs(to64(d) - e) <= ((1 + U32) ** 4 - 1) * np.abs(e))


@pytest.mark.parametrize("vocab", [131072, 152064])
def test_head_of_a_large_vocabulary(vocab):
    """An 8-bit head against a teacher, forward and backward: the input
    gradient's depth is the vocabulary."""
    tokens, dim, k = 48, 128, 16
    g = torch.Generator(DEV).manual_seed(7)
    W = (0.1 * torch.randn((vocab, dim), generator=g, device=DEV)).to(BF)
    x = torch.randn((tokens, dim), generator=g, device=DEV).to(BF)
    e = lambda *s, d=F32: torch.empty(s, dtype=d, device=DEV)  # noqa: E731
    q = lambda r, c: (ouo.int8_empty(r, c), e(r))  # noqa: E731
    wq, wt, xq, xt, dq, dt = (q(*s) for s in ((vocab, dim), (dim, vocab), (tokens, dim),
                                              (dim, tokens), (tokens, vocab), (vocab, tokens)))
    teacher = torch.randn((tokens, k), generator=g, device=DEV)
    idx = torch.randint(0, vocab, (tokens, k), generator=g, device=DEV).to(torch.int32)
    S, dS, loss, lse = e(tokens, vocab, d=BF), e(tokens, vocab, d=BF), e(tokens), e(tokens)
    dx, dW = e(tokens, dim, d=BF), e(vocab, dim)
    ouo.quantize_int8(W, *wq)
    ouo.quantize_int8(W, *wt, transpose=True)
    ouo.quantize_int8(x, *xq)
    ouo.quantize_int8(x, *xt, transpose=True)
    ouo.int8_matmul(*xq, *wq, S)
    ouo.distill_loss(S, teacher, idx, loss, lse)
    ouo.distill_loss_backward(S, teacher, idx, lse, torch.ones_like(loss), dS)
    ouo.quantize_int8(dS, *dq)
    ouo.quantize_int8(dS, *dt, transpose=True)
    ouo.int8_matmul(*dq, *wt, dx)
    ouo.int8_matmul(*dt, *xt, dW)
    bf = (1 + 2.0 ** -8) * (1 + U32) ** 3 - 1
    for out, (a, sa), (b, sb), tol in ((S, xq, wq, bf), (dx, dq, wt, bf),
                                       (dW, dt, xt, (1 + U32) ** 4 - 1)):
        want = _exact_product(a, sa, b, sb)
        assert np.all(np.abs(to64(out) - want) <= tol * np.abs(want))
    # 8-bit operands: half a step of each, summed over the vocabulary
    d, w = to64(dS), to64(W)
    a, b = np.abs(d).max(1) / 254, np.abs(w).max(0) / 254
    slack = np.abs(d).sum(1)[:, None] * b + a[:, None] * np.abs(w).sum(0) + vocab * a[:, None] * b
    want = d @ w
    assert np.all(np.abs(to64(dx) - want) <= slack * 1.001 + 2.0 ** -8 * np.abs(want))
    assert torch.isfinite(loss).all() and (loss > 0).all()


# ------------------------------------------- the gradient, value by value


@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("rows,vocab,k", [
    (1, 50001, 20), (33, 4099, 64), (70, 2048, 7), (2, 131072, 128), (9, 32768, 1024),
    (300, 515, 33), (700, 64, 5), (1300, 20000, 16)])
def test_distill_gradient_value_by_value(rows, vocab, k, tau, dtype, out):
    g = torch.Generator(DEV).manual_seed(vocab)
    s = (torch.randn((rows, vocab), generator=g, device=DEV) * 3).to(dtype)
    t = torch.randn((rows, k), generator=g, device=DEV) * 2 + 5
    idx = torch.randint(0, vocab, (rows, k), generator=g, device=DEV).to(torch.int32)
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ouo.distill_loss(s, t, idx, loss, lse, temperature=tau)
    dl = torch.randn(rows, generator=g, device=DEV)
    ds = torch.empty((rows, vocab), dtype=out, device=DEV)
    ouo.distill_loss_backward(s, t, idx, lse, dl, ds, temperature=tau)
    # in float64 on the device: the oracle's sums one by one would take minutes
    x = s.double() / tau
    q = torch.exp(x - lse.double()[:, None])
    lp = torch.log_softmax(t.double() / tau, 1)
    p = torch.zeros_like(q).scatter_add_(1, idx.long(), lp.exp())
    scale = (dl.double() * tau)[:, None]
    e = scale * (q - p)
    z = (x.abs().max() + lse.abs().max()).item()
    zt = (t.abs().max() / tau).item()
    # q's exponent: 1 / tau, the fused product, log2(e) (2); the exponential (2
    # ulp); g and its product.  p's: two in the difference by tau, 1 / tau; the
    # exponential, its sum and quotient, equal indices
    eq = (4 * z + 8) * U32 * q
    ep = (6 * zt + k / 128 + 52) * U32 * p
    tol = scale.abs() * (eq + ep + 2.0 ** -126) + ({BF: 2.0 ** -8, F32: U32}[out] + U32) * e.abs()
    assert bool(((ds.double() - e).abs() <= tol).all())
