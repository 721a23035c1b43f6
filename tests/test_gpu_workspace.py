"""Calls with a workspace on several streams and in several graphs at once."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_attention_q8 import _case

pytestmark = pytest.mark.gpu

SHAPE = (1, 2, 8, 64, 512)      # T, H, G, D, K: joined by a launch


def _calls(dev, n):
    out = []
    for i in range(n):
        q, c, s, bt, ctx, dtype, _ = _case(*SHAPE, "e4m3", [65536 - 1000 * i, 60000], 200 + i, pages=1500)
        for x in c:
            x[(x & 0x7F) == 0x7F] = 0x31
        out.append([x.to(dev) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)])
    return out


def test_two_graphs_replayed_at_once(cuda_device):
    """Two graphs captured one after the other on PyTorch's own capture stream,
    replayed on two streams at once beside eager calls on a third."""
    dev = cuda_device
    assert bsa.bsa_attention_q8_workspace_bytes(*SHAPE) > 0
    calls = _calls(dev, 3)
    ref = [bsa.bsa_sparse_decode_attention_q8(*a) for a in calls]
    torch.cuda.synchronize()
    outs = [torch.empty_like(r) for r in ref]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, args, out in zip(graphs, calls, outs):
        with torch.cuda.graph(graph):
            for _ in range(8):
                bsa.bsa_sparse_decode_attention_q8(*args, out=out)
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
            for _ in range(8):
                bsa.bsa_sparse_decode_attention_q8(*calls[2], out=outs[2])
        torch.cuda.synchronize()
        for o, r in zip(outs, ref):
            assert torch.equal(o, r)


def test_a_callers_workspace_is_used_within_its_bytes(cuda_device):
    """Full of old bytes, on a side stream: the same bits, written up to the bytes
    asked for and not behind them; less, or misaligned, is refused."""
    dev = cuda_device
    need = bsa.bsa_attention_q8_workspace_bytes(*SHAPE)
    assert need > 0
    args, = _calls(dev, 1)
    ref = bsa.bsa_sparse_decode_attention_q8(*args)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream(dev)
    with torch.cuda.stream(stream):
        got = [bsa.bsa_sparse_decode_attention_q8(*args, workspace=ws[:need]) for _ in range(2)]
    stream.synchronize()
    assert all(torch.equal(g, ref) for g in got)
    assert (ws[need:] == 0xFF).all() and (ws[:need] != 0xFF).any()
    for bad in (ws[:need - 1], ws[16:need + 16], torch.empty(0, dtype=torch.uint8, device=dev)):
        with pytest.raises(bsa.BsaError) as e:
            bsa.bsa_sparse_decode_attention_q8(*args, workspace=bad)
        assert e.value.status == -5
