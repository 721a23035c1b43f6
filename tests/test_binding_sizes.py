"""Sizes past 32 bits in the cache operators' arguments (meta tensors: no memory,
and nothing can be launched)."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from block_sparse_attention_topk_gb300 import build


def _meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("name,value", [
    ("inv_freq", _meta(2**31 + 32)), ("inv_freq", _meta(2**30)), ("positions", _meta(2**32 + 1, 4, dtype=torch.int32)),
])
def test_counts_that_do_not_fit(name, value):
    build.build()
    x = _meta(4, 2, 64, dtype=torch.bfloat16)
    good = dict(positions=_meta(4, dtype=torch.int32), inv_freq=_meta(32))
    with pytest.raises(ValueError, match=f"{name} .*long|{name} .*axes"):
        bsa.bsa_rope(x, **{**good, name: value})
