"""The 8-bit attention when waits inside it run out: the copies of each CTA stop
after some stages, and the waits for them have a limit of 2 ms.  Nothing on the
GPU goes wrong; each output is right or NaN, and the status word says so."""
import ctypes

import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_attention_q8 import _case

pytestmark = pytest.mark.gpu


@pytest.fixture
def stall(cuda_device):
    fn = bsa.lib().bsa_attention_q8_stall
    fn.argtypes, fn.restype = [ctypes.c_uint32, ctypes.c_uint64], None
    word = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    bsa.bsa_set_status_word(word)
    yield fn
    fn(2**32 - 1, 0)
    bsa.bsa_set_status_word(None)


@pytest.mark.parametrize("T,H,G,D,K,joined", [
    (300, 2, 4, 64, 6, None), (700, 1, 8, 128, 20, None), (200, 2, 16, 128, 9, None), (310, 1, 3, 256, 8, None),
    (1, 1, 8, 128, 16, "cluster"), (3, 1, 12, 64, 8, "cluster"), (2, 1, 3, 256, 2, "cluster"),
    (1, 2, 8, 64, 512, "launch"), (1, 1, 16, 128, 1024, "launch"),
])
def test_waits_that_run_out(cuda_device, stall, T, H, G, D, K, joined):
    dev = cuda_device
    ctx = [K * 128 - 37 * i % (K * 64) for i in range(T * H)]
    q, c, s, bt, ctx, dtype, _ = _case(T, H, G, D, K, "e4m3", ctx, 300 + D, pages=1200)
    for x in c:
        x[(x & 0x7F) == 0x7F] = 0x31
    args = [x.to(dev) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)]
    assert (bsa.bsa_attention_q8_workspace_bytes(T, H, G, D, K) > 0) == (joined == "launch")
    ref = bsa.bsa_sparse_decode_attention_q8(*args)
    assert bsa.bsa_read_status() == 0 and torch.isfinite(ref).all()
    out = torch.empty_like(ref)
    finished = []
    for stages in (0, 1, 2, 3, 5, 9, 14, 27, 50, 10000):
        stall(stages, 2000000)
        out.fill_(7.0)
        bsa.bsa_sparse_decode_attention_q8(*args, out=out)
        status = bsa.bsa_read_status()
        nan = torch.isnan(out)
        assert torch.equal(torch.where(nan, ref, out), ref), stages
        assert status == (bsa.BSA_STATUS_TIMEOUT if nan.any() else 0), stages
        finished.append(int((~nan).sum()))
    assert finished[0] == 0 and finished[-1] == ref.numel()
    assert finished == sorted(finished)
    stall(2**32 - 1, 0)
    assert torch.equal(bsa.bsa_sparse_decode_attention_q8(*args, out=out), ref)
    assert bsa.bsa_read_status() == 0
