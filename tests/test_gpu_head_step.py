"""GPU test of the benchmark's training step of an 8-bit head against a
teacher (norm, products, distillation, gradients, Dion3 step): it runs, also
with a vocabulary whose input gradient is a deep product, and moves the
weight."""
import json
import types

import pytest
import torch

import bench

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,m,n", [(96, 640, 256), (33, 1000, 136), (16, 131200, 64)])
def test_head_step_runs(tokens, m, n):
    step, ops = bench.head8_step(tokens, m, n, torch.device("cuda", 0), k=8)
    assert ops == 6 * tokens * m * n
    held = {k: c.cell_contents for k, c in zip(step.__code__.co_freevars, step.__closure__)}
    before = held["W"].clone()
    step()
    first = held["loss"].clone()
    assert torch.isfinite(first).all() and torch.isfinite(held["dX"]).all()
    changed = (held["W"] != before).any(1).sum().item()
    assert 0 < changed <= m // 8 + 1
    # the 8-bit copies are those of the weight as it is now
    q, s = held["wq"]
    assert ((q * s[:, None] - held["W"].float()).abs() <= 0.51 * s[:, None]).all()
    for _ in range(2):
        step()
    assert torch.isfinite(held["loss"]).all() and torch.isfinite(held["W"]).all()


@pytest.mark.parametrize("case", [
    dict(op="rms", rows=5, cols=64, dtype="bf16", residual=True, int8=True, stream="f32"),
    dict(op="rms_bwd", rows=5, cols=64, dtype="bf16", stream="f32"),
    dict(op="mm", m=5, n=16, k=64, dtype="bf16", unaligned=True)])
def test_timing_of_a_call_runs(case, capsys):
    bench.run_tokens(types.SimpleNamespace(case=[json.dumps(case)]))
    line = json.loads(capsys.readouterr().out)
    assert line["case"] == case and line["us"] > 0 and line["us_load"] > 0
