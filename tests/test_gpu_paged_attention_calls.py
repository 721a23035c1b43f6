"""Paged attention in several graphs and streams at once, in a caller's workspace, on
views at 16 bytes, and when waits inside it run out."""
import ctypes

import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu


def _case(i, fmt="bf16"):
    case = Case("varlen", (0, [(300 + i, 900), (5, 2000 - i), (40, 0)]), 2, 6, 128, fmt, seed=100 + i)
    case.c = [x.float().nan_to_num(0.5).to(x.dtype) for x in case.c]
    return case


def test_two_graphs_replayed_at_once(cuda_device):
    dev = cuda_device
    calls = [_case(i, ("bf16", "e4m3", "bf16")[i]).args(dev) for i in range(3)]
    ref = [fn(*args, **more) for fn, args, more in calls]
    torch.cuda.synchronize()
    outs = [torch.empty_like(r) for r in ref]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, (fn, args, more), out in zip(graphs, calls, outs):
        with torch.cuda.graph(graph):
            for _ in range(4):
                fn(*args, **more, out=out)
    streams = [torch.cuda.Stream(dev) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            fn, args, more = calls[2]
            for _ in range(4):
                fn(*args, **more, out=outs[2])
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            assert torch.equal(o, r)


def test_a_callers_workspace_is_used_within_its_bytes(cuda_device):
    dev = cuda_device
    fn, args, more = _case(0).args(dev)
    T, H, G, D = args[0].shape
    need = bsa.bsa_paged_attention_workspace_bytes(T, H, G, D)
    assert need > 0 and need == bsa.bsa_paged_attention_workspace_bytes(T, H, G, D, dev)
    ref = fn(*args, **more)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream(dev)
    with torch.cuda.stream(stream):
        got = [fn(*args, **more, workspace=ws[:need]) for _ in range(2)]
    stream.synchronize()
    assert all(torch.equal(g, ref) for g in got)
    assert (ws[need:] == 0xFF).all() and (ws[:need] != 0xFF).any()
    for bad in (ws[:need - 1], ws[16:need + 16], torch.empty(0, dtype=torch.uint8, device=dev)):
        with pytest.raises(bsa.BsaError) as e:
            fn(*args, **more, workspace=bad)
        assert e.value.status == -5


def test_outputs_at_16_bytes(cuda_device):
    """An output that is 16-byte and not 32-byte aligned: the same bits, and nothing around it."""
    dev = cuda_device
    for fmt in ("bf16", "e5m2"):
        fn, args, more = _case(1, fmt).args(dev)
        ref = fn(*args, **more)
        buf = torch.full((ref.numel() + 16,), 3.0, dtype=torch.bfloat16, device=dev)
        out = buf[8:8 + ref.numel()].view(ref.shape)
        assert out.data_ptr() % 32 == 16
        fn(*args, **more, out=out)
        assert torch.equal(out, ref) and (buf[:8] == 3).all() and (buf[-8:] == 3).all()


def test_version_counters_move(cuda_device):
    fn, args, more = _case(2).args(cuda_device)
    out = torch.empty_like(args[0])
    before = out._version
    fn(*args, **more, out=out)
    assert out._version > before and args[0]._version == 0


@pytest.fixture
def stall(cuda_device):
    fn = bsa.lib().bsa_paged_attention_stall
    fn.argtypes, fn.restype = [ctypes.c_uint32, ctypes.c_uint64], None
    word = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    bsa.bsa_set_status_word(word)
    yield fn
    fn(2**32 - 1, 0)
    bsa.bsa_set_status_word(None)


@pytest.mark.parametrize("form,rows,H,G,D,fmt", [
    ("varlen", (0, [(600, 1500), (3, 4000)]), 2, 8, 128, "bf16"), ("varlen", (0, [(300, 900)]), 2, 8, 64, "e4m3"),
    ("decode", (1, [3000 + 10 * i for i in range(200)]), 2, 8, 128, "e5m2"), ("decode", (2, [900] * 100), 2, 4, 64, "bf16"),
    ("varlen", (0, [(200, 1000)]), 2, 5, 256, "bf16"), ("varlen", (0, [(100, 1000)]), 2, 5, 256, "e4m3"),
])
def test_waits_that_run_out(cuda_device, stall, form, rows, H, G, D, fmt):
    """The copies of each CTA stop after some stages, and waits have a limit of 2 ms.  Nothing on
    the GPU goes wrong; each output is right or NaN, and the status word says so."""
    case = Case(form, rows, H, G, D, fmt, seed=7)
    case.c = [x.float().nan_to_num(0.5).to(x.dtype) for x in case.c]
    fn, args, more = case.args(cuda_device)
    ref = fn(*args, **more)
    assert bsa.bsa_read_status() == 0 and torch.isfinite(ref).all()
    out = torch.empty_like(ref)
    finished = []
    for stages in (0, 1, 2, 3, 5, 9, 14, 27, 50, 100000):
        stall(stages, 2000000)
        out.fill_(7.0)
        fn(*args, **more, out=out)
        status = bsa.bsa_read_status()
        nan = torch.isnan(out)
        assert torch.equal(torch.where(nan, ref, out), ref), stages
        assert status == (bsa.BSA_STATUS_TIMEOUT if nan.any() else 0), stages
        finished.append(int((~nan).sum()))
    assert finished[-1] == ref.numel()
    stall(2**32 - 1, 0)
    assert torch.equal(fn(*args, **more, out=out), ref)
    assert bsa.bsa_read_status() == 0
