"""CPU checks of where the bindings take their own buffers from: a call on
another stream uses that stream's pool, since a block of the current stream's
pool may still be in use there."""
import contextlib
import types

import pytest
import torch

from orthonormalized_update_optimizers_b200 import binding, tokens


class _Stream:
    device = types.SimpleNamespace(index=-1)  # what a host tensor's get_device says


@pytest.fixture
def taken(monkeypatch):
    """Sizes of torch.empty's buffers and the stream that was current."""
    now, log, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def take(n, *a, **kw):
        log.append((n, now[-1]))
        return empty(n, dtype=kw.get("dtype"))

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", take)
    return log


def test_token_workspace_belongs_to_the_stream_that_uses_it(taken):
    s = _Stream()
    out = tokens._workspace(1024, None, -1, s)
    assert taken == [(1024, s)]
    # the tensor is handed out with its address, so that it lives until the launch
    assert out[0].data_ptr() == out[1] and out[2] == 1024
    tokens._workspace(512, None, -1, None)
    assert taken[1:] == [(512, None)]
    tokens._workspace(0, None, -1, s)
    assert len(taken) == 2


def test_token_workspace_of_another_device_is_refused_first(taken):
    with pytest.raises(ValueError, match="the stream is on"):
        tokens._workspace(1024, None, 0, _Stream())
    assert not taken


def test_optimizer_workspace_belongs_to_the_stream_that_uses_it(taken):
    s = _Stream()
    binding._workspace(4096, torch.device("cpu"), None, s)
    binding._workspace(4096, torch.device("cpu"), None, None)
    assert taken == [(4096, s), (4096, None)]
