"""CPU checks of the token operators' limits; nothing is launched (the
pointers are fake)."""
import ctypes

import pytest
import torch

from orthonormalized_update_optimizers_b200 import _lib as L
from orthonormalized_update_optimizers_b200 import build as B
from orthonormalized_update_optimizers_b200 import tokens

BAD, UNSUP, NODEV = -1, -2, -5


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def _m(rows, cols, ptr=0x10000):
    return (L.OuoMat * 1)(L.OuoMat(ptr, rows, cols, cols))


def _mm(fn, depth, d=None, scale=0x20000):
    v = (ctypes.c_void_p * 1)(scale)
    return fn(_m(4, depth), v, _m(6, depth, 0x4000000), v, d or _m(4, 6, 0x9000000), L.OUO_BF16, 1,
              None, None)


def test_deep_products_are_taken_up_to_their_limit(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for depth in (0, 64, L.OUO_INT8_MAX_DEPTH, 131072, 152064, L.OUO_INT8_MAX_DEEP):
        assert _mm(lib.int8_matmul_deep, depth) == NODEV


def test_deeper_products_are_refused(lib):
    assert _mm(lib.int8_matmul_deep, L.OUO_INT8_MAX_DEEP + 1) == UNSUP
    assert b"depth 1047553 above 1047552" in lib.ouo_last_error()
    assert _mm(lib.int8_matmul_deep, 152064, d=_m(4, 7, 0x9000000)) == BAD
    assert _mm(lib.int8_matmul_deep, 152064, scale=None) == BAD
    # no sum of a piece leaves 32 bits, whatever the integers
    assert L.OUO_INT8_MAX_DEPTH * 128 * 128 < 2 ** 31


class _OnDevice0(torch.Tensor):
    """A host tensor that says it is on device 0."""

    def get_device(self):
        return 0


@pytest.mark.parametrize("depth,entry", [(64, "int8_matmul"), (131071, "int8_matmul"),
                                         (131072, "int8_matmul_deep"),
                                         (152064, "int8_matmul_deep")])
@pytest.mark.parametrize("batch", [False, True])
def test_the_binding_chooses_by_depth(monkeypatch, depth, entry, batch):
    called = []
    monkeypatch.setattr(tokens, "_run", lambda name, *a: called.append(name))

    def t(*shape, dtype=torch.int8):
        return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice0)

    a, b, d = t(2, depth), t(3, depth), t(2, 3, dtype=torch.float32)
    sa, sb = t(2, dtype=torch.float32), t(3, dtype=torch.float32)
    if batch:
        tokens.int8_matmul([t(2, 8), a], [sa, sa], [t(3, 8), b], [sb, sb], [d, d])
    else:
        tokens.int8_matmul(a, sa, b, sb, d)
    assert called == [entry]
