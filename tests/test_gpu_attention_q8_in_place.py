"""The 8-bit attention with the queries' memory as its output."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_attention_q8 import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,G,D,K", [(700, 2, 8, 128, 5), (300, 3, 1, 64, 7), (3, 1, 12, 64, 8), (1, 2, 8, 64, 512)])
def test_out_is_q(cuda_device, T, H, G, D, K):
    """One CTA per row, a cluster's, and joined by a launch: the same bits."""
    q, c, s, bt, ctx, dtype, _ = _case(T, H, G, D, K, "e4m3", [K * 128 - i % 300 for i in range(T * H)], 500 + D, pages=900)
    for x in c:
        x[(x & 0x7F) == 0x7F] = 0x31
    args = [x.to(cuda_device) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)]
    ref = bsa.bsa_sparse_decode_attention_q8(*args)
    assert bsa.bsa_sparse_decode_attention_q8(*args, out=args[0]) is args[0]
    torch.cuda.synchronize()
    assert torch.equal(args[0], ref)
