"""Who shares the package's workspaces, without a GPU: CPU tensors stand in for
device memory, the current stream and the capture are given."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa


@pytest.fixture
def places(monkeypatch):
    """The current stream and whether it is being captured, as a dict to set."""
    state = {"stream": 1, "capturing": False}
    monkeypatch.setattr(bsa, "_stream", lambda device: state["stream"])
    monkeypatch.setattr(bsa, "_capturing", lambda device: state["capturing"], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(bsa, "_ws_cache", {})
    return state


CPU = torch.device("cpu")


def test_captured_calls_share_no_workspace(places):
    """Graphs replay on any stream, whatever stream captured them: each captured
    call has memory of its own, apart from the eager calls' of that stream."""
    eager = bsa._workspace(CPU, 256)
    places["capturing"] = True
    a, b = bsa._workspace(CPU, 256), bsa._workspace(CPU, 256)
    places["capturing"] = False
    again = bsa._workspace(CPU, 256)
    assert again.data_ptr() == eager.data_ptr()
    assert len({x.data_ptr() for x in (eager, a, b)}) == 3


def test_captured_workspaces_go_with_their_graph(places):
    """Nothing outside the capture's memory pool holds a captured workspace."""
    import gc
    import weakref
    places["capturing"] = True
    ref = weakref.ref(bsa._workspace(CPU, 1024))
    gc.collect()
    assert ref() is None


def test_eager_calls_share_along_a_stream(places):
    a = bsa._workspace(CPU, 256)
    assert bsa._workspace(CPU, 128).data_ptr() == a.data_ptr()
    places["stream"] = 2
    assert bsa._workspace(CPU, 256).data_ptr() != a.data_ptr()
    places["stream"] = 1
    assert bsa._workspace(CPU, 512).numel() >= 512
    assert bsa._workspace(CPU, 0) is None
