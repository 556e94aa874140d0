"""CPU tests of how the calls tell autograd what they have written."""
import pytest

torch = pytest.importorskip("torch")


def test_versions_advance():
    from gated_deltanet_chunked_varlen_amd import api
    a, b = torch.zeros(3), torch.zeros((4, 2))
    view = b[1:]
    with torch.inference_mode():
        inf = torch.zeros(2)
    api._advance_versions(a, None, view, inf)
    assert a._version == 1 and b._version == 1 and view._version == 1
    api._advance_versions()
    api._advance_versions(None)
    with pytest.raises((TypeError, ValueError)):
        api._advance_versions(3)
    w = torch.ones(3, requires_grad=True)
    y = (w * a).sum()
    api._advance_versions(a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
