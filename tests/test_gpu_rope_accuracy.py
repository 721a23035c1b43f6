"""The rotation's error in norm, fp32.

Relative to the rows, with errors taken as evenly spread: the result's rounding
2.5e-8, the rounded one of its two products 1.2e-8, cosines and sines within one unit
in the last place 2.4e-8, the angle's 24 bits on an eighth of a turn at most 1.0e-8
(on half a turn it would be 4.1e-8): 3.8e-8 in all.  A fifth is left for their
distributions."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_error_in_norm(cuda_device, interleaved, inverse):
    g = torch.Generator().manual_seed(1)
    T, H, D = 2000, 2, 128
    x = torch.randn((T, H, D), generator=g)
    pos = torch.randint(-(1 << 20), 1 << 20, (1, T), generator=g).to(torch.int32)
    inv = (1e4 ** (-torch.arange(64) / 64)).float()
    want = oracle.rope(x.double().numpy(), pos.numpy(), inv.numpy(), None, interleaved, inverse)
    got = bsa.bsa_rope(x.to(cuda_device), pos[0].to(cuda_device), inv.to(cuda_device), interleaved=interleaved, inverse=inverse)
    torch.cuda.synchronize()
    assert np.linalg.norm(got.double().cpu().numpy() - want) <= 4.6e-8 * np.linalg.norm(want)
