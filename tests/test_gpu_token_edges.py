"""GPU tests of the token-matrix operators where they are easiest to get
wrong."""
import numpy as np
import pytest
import torch

import orthonormalized_update_optimizers_b200 as ouo

from ._util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


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
@pytest.mark.parametrize("copies", [1, 24])  # 24: past the 3 MB of the one-read transposition
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
