"""CPU test of where a differentiable call looks for a graph capture."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import recurrence  # noqa: E402


def test_capture_is_looked_for_on_the_tensors_device(monkeypatch):
    """Device 1 captures while device 0 is the current one."""
    current = [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == 1)

    def on(i):
        return types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", i))

    assert not recurrence._capturing(on(0)) and recurrence._capturing(on(1))
    assert current == [0]
    assert not recurrence._capturing(torch.zeros(2))
