"""CPU pins of the token-matrix oracle: gradients against differences,
closed forms, padding."""
import numpy as np
import pytest

from oracle import tokens as ot


def _num_grad(f, x, d=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += d
        b[i] -= d
        g[i] = (f(a) - f(b)) / (2 * d)
    return g


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_is_the_differences(tau):
    r = np.random.default_rng(0)
    s, t = r.normal(size=(4, 11)), r.normal(size=(4, 5)) * 2
    idx = np.array([[0, 3, 7, 2, 10], [1, 1, 4, -1, 5], [-1] * 5, [9, 11, 2, 3, -7]])
    dl = r.normal(size=4)
    lse = ot.distill_loss(s, t, idx, tau)[1]
    num = _num_grad(lambda x: float(np.sum(dl * ot.distill_loss(x, t, idx, tau)[0])), s)
    # central differences at 1e-5: error ~ d^2 f''' + 2^-53 |f| / d ~ 1e-9
    assert np.abs(ot.distill_grad(s, t, idx, lse, dl, tau) - num).max() < 1e-8


def test_distill_of_the_same_distribution_is_zero():
    r = np.random.default_rng(1)
    s = r.normal(size=(3, 8))
    idx = np.tile(np.arange(8), (3, 1))
    loss, lse = ot.distill_loss(s, s, idx, 1.0)
    assert np.abs(loss).max() < 1e-14
    assert np.abs(ot.distill_grad(s, s, idx, lse, np.ones(3), 1.0)).max() < 1e-15


def test_rms_gradient_is_the_differences():
    r = np.random.default_rng(2)
    h, w, dy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=(3, 7))
    rstd = ot.rms_norm(h, w, 1e-3)[1]
    dx, dw = ot.rms_norm_grad(dy, h, w, rstd)
    assert np.abs(dx - _num_grad(lambda x: float(np.sum(dy * ot.rms_norm(x, w, 1e-3)[0])), h)).max() < 1e-8
    assert np.abs(dw - _num_grad(lambda x: float(np.sum(dy * ot.rms_norm(h, x, 1e-3)[0])), w)).max() < 1e-8


def test_quantize_bounds():
    r = np.random.default_rng(3)
    x = r.normal(size=(5, 40))
    x[2] = 0
    q, scale = ot.quantize(x)
    assert np.abs(q).max() <= 127 + 1e-12 and scale[2] == 0 and not q[2].any()
    assert np.allclose(q * scale[:, None], x, rtol=1e-14)
    assert ot.quantize(np.zeros((2, 0)))[1].tolist() == [0, 0]
