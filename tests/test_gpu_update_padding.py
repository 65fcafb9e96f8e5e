"""GPU test: the low-rank step's in-place updates leave what stands beside
the matrices alone (a matrix may be some columns of a wider one)."""
import numpy as np
import pytest
import torch

import orthonormalized_update_optimizers_b200 as ouo
from orthonormalized_update_optimizers_b200 import synth
from oracle import dion as odion

from ._util import TOL_BF16, rel_fro, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

# odd and ragged column counts, rows within and past one tile
SHAPES = [(70, 33), (130, 65), (256, 129), (300, 514), (40, 1001), (256, 128)]


def _inside(rows, cols, dtype, beside, fill=None):
    """A rows x cols matrix inside a wider one that holds `beside` elsewhere,
    its rows on 16-byte boundaries."""
    buf = torch.full((rows + 2, (cols + 23) // 16 * 16 + 16), beside, device=DEV).to(dtype)
    v = buf[1:rows + 1, 8:8 + cols]
    if fill is not None:
        v.copy_(fill)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[1:rows + 1, 8:8 + cols] = False
    return buf, v, rest


@pytest.mark.parametrize("mode", [odion.COLNORM, odion.QR])
@pytest.mark.parametrize("w_dtype", [BF, F32])
@pytest.mark.parametrize("grouped", [False, True])
def test_low_rank_step_beside_other_columns(mode, w_dtype, grouped):
    r, lr = 16, 0.01
    p = ouo.dion_params(rank=r, lr=lr, norm_mode="qr" if mode == odion.QR else "colnorm")
    got = []
    for beside in (0.0, 77.0):
        sets = []
        for i, (m, n) in enumerate(SHAPES):
            G = synth.lowrank_plus_noise(m, n, min(32, m, n), 0.02, 50 + i, BF, DEV)
            M = _inside(m, n, F32, beside, torch.zeros((m, n), device=DEV))
            W0 = synth.gaussian((m, n), 90 + i, 0.02, w_dtype, DEV)
            W = _inside(m, n, w_dtype, beside, W0)
            q0 = odion.orth(synth.dion_q0(n, r, 1).double().numpy()).astype(np.float32)
            sets.append((M, G, torch.tensor(q0.T.copy(), device=DEV), W, W0, q0))
        # Q_state's rows on 16-byte boundaries too
        Q = [_inside(r, s[2].shape[1], F32, beside, s[2]) for s in sets]
        for k in [slice(None)] if grouped else [slice(i, i + 1) for i in range(len(sets))]:
            ouo.dion_lowrank_step([s[0][1] for s in sets[k]], [s[1] for s in sets[k]],
                                  [q[1] for q in Q[k]], [s[3][1] for s in sets[k]], p)
        for s, q in zip(sets, Q):
            for buf, _, rest in (s[0], s[3], q):
                assert bool((buf[rest].float() == beside).all()), "written outside the matrix"
        got.append([(s[0][1].clone(), q[1].clone(), s[3][1].clone()) for s, q in zip(sets, Q)])
    # whatever stands beside them, the results are the same
    for a, b in zip(*got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for s, (M, _, W) in zip(sets, got[0]):
        ref = odion.dion_step(np.zeros(M.shape, np.float32), to64(s[1]), s[5].astype(np.float64),
                              to64(s[4]), 0.95, lr, 1.0, mode)
        assert rel_fro(to64(M), ref["M"]) <= TOL_BF16
        err = np.linalg.norm(to64(W) - ref["W"])
        # the update's error, and one rounding of the weights to their type
        rnd = (2.0 ** -8 if w_dtype == BF else 2.0 ** -24) * np.linalg.norm(ref["W"])
        assert err <= TOL_BF16 * np.linalg.norm(ref["W"] - to64(s[4])) + rnd
