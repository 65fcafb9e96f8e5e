"""CPU check of the kernels' sources: every wait has a limit, and a wait that
ran out is heard of (its result is looked at, so that the status is set)."""
import glob
import os
import re

from orthonormalized_update_optimizers_b200 import build as B


def _statements(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [" ".join(t.split()) for t in re.split(r"[;{}]", text)]


def test_no_wait_runs_out_unheard():
    waits = unheard = 0
    for path in sorted(glob.glob(os.path.join(B.CSRC, "*.cu"))):
        for t in _statements(path):
            if "ptx::mbar_wait" not in t:
                continue
            waits += 1
            # a bare call, or one behind a condition or a loop of its own
            if re.match(r"(if \([^!]*\) |for \(.*\) )*ptx::mbar_wait", t):
                # copies in flight are given 100 ms after a timeout that was reported
                if "100000000ull" not in t:
                    unheard += 1
                    print(os.path.basename(path), t)
    assert waits > 10 and unheard == 0


def test_every_wait_has_a_limit():
    """Nothing but the two bounded waits polls a barrier."""
    with open(os.path.join(B.CSRC, "umma.cuh")) as f:
        text = f.read()
    assert len(re.findall(r"mbar_try_wait\(bar, parity\)", text)) == 3
    for path in glob.glob(os.path.join(B.CSRC, "*.cu")):
        with open(path) as f:
            assert "mbar_try_wait" not in f.read(), path
