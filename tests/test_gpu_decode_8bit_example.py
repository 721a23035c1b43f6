"""The decode example: append, select, table and attention over the 8-bit cache
together, against the same loop over a bf16 cache.

Tolerance.  The example's values are N(0, 1).  A value's code is off by at most
2^-4 of it, uniformly on average: 2^-4 / sqrt(3) / (about 1.4) = 0.026 relative
rms.  Averaged over the context, the values' part of the output's error stays
0.026 relative; a key's error moves a score by 0.026 rms (scores are N(0, 1)),
so each probability by 0.026, which adds as much again: 0.026 sqrt(2) = 0.037,
and subnormals and the two roundings to bf16 below 0.005.  0.06 bounds it."""
import pytest
import torch

from examples.decode_8bit_cache import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,H,K", [(128, 8, 2, 16), (64, 4, 1, 8), (256, 3, 2, 16)])
def test_decode_loop_over_the_8_bit_cache(cuda_device, D, G, H, K):
    outs = run(steps=5, prompts=(1500, 700, 33), H=H, G=G, D=D, K=K, seed=D)
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.isfinite(a).all()
        assert float((a.float() - b).norm() / b.norm()) <= 0.06
