"""CPU tests of the workspaces kept per stream: the recurrence's beside the
prefill's, the least recently used dropped first."""
import threading

import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_chunked_varlen_amd import _launch, api  # noqa: E402


@pytest.fixture(autouse=True)
def _cpu_memory(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(_launch, "_memory", lambda index, need: torch.empty(need,
                                                                            dtype=torch.uint8))
    api.clear_workspace_cache()
    yield
    api.clear_workspace_cache()


def test_kept_grown_and_cleared():
    ws = _launch._workspace(0, 7, 100)
    assert _launch._workspace(0, 7, 50) is ws
    big = _launch._workspace(0, 7, 200)
    assert big.numel() >= 200 and _launch._workspace(0, 7, 100) is big
    assert _launch._workspace(0, 8, 100) is not big
    assert _launch._workspace(1, 7, 100) is not big
    api.clear_workspace_cache()
    assert _launch._workspace(0, 7, 100) is not big


def test_the_least_recently_used_goes_first():
    most = api._WS_CACHE_MAX
    hot = _launch._workspace(0, 0, 10)
    for s in range(1, 3 * most):
        _launch._workspace(0, s, 10)
        assert _launch._workspace(0, 0, 10) is hot
    assert len(_launch._ws_cache) == most


def test_the_prefill_keeps_its_own(monkeypatch):
    """Recurrence calls on many streams leave the prefill's workspaces alone."""
    kept = [api.cached_workspace("cpu", s, 10) for s in range(api._WS_CACHE_MAX)]
    for s in range(2 * api._WS_CACHE_MAX):
        _launch._workspace(0, s, 10)
    for s, ws in enumerate(kept):
        assert api.cached_workspace("cpu", s, 10) is ws


def test_threads():
    wrong = []

    def work(k):
        for i in range(400):
            try:
                if _launch._workspace(0, (k * 31 + i) % 90, 10 + i).numel() < 10 + i:
                    wrong.append(i)
                if i % 50 == 0:
                    api.clear_workspace_cache()
            except Exception as e:  # noqa: BLE001
                wrong.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
