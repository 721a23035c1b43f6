"""Appends of more rows than stay in registers, with every kind of pair, against
the 64-bit oracle within the tolerance of tests/test_gpu_append.py."""
import pytest
import torch

from tests.test_gpu_append import TYPES, _compare, _setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(TYPES))
@pytest.mark.parametrize("T", [2700, 5300])
@pytest.mark.parametrize("H,Hq,D,rot,inter,axes", [
    (2, 3, 64, 64, True, 1), (1, 2, 80, 62, True, 3), (2, 1, 64, 30, False, 1), (1, 3, 128, 106, False, 3),
    (1, 1, 256, 2, False, 2), (2, 2, 64, 64, False, 3), (1, 2, 48, 40, False, 2), (3, 0, 32, 26, False, 1),
])
def test_append_long_calls(cuda_device, fmt, T, H, Hq, D, rot, inter, axes):
    lens = [449] * (T // 449) + [T % 449]
    pre = [(7 * i) % 60 for i in range(len(lens))]
    qkv, table, caches, _, kind = _setup(T + 5, H, Hq, D, len(lens), 4, fmt, T + D + rot)
    cu = torch.tensor([2] + lens).cumsum(0).to(torch.int32)
    g = torch.Generator().manual_seed(T)
    positions = axis = None
    if axes > 1:
        positions = torch.randint(0, 100000, (axes, T + 5), generator=g, dtype=torch.int32)
        axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    _compare(cuda_device, "varlen", qkv, H, Hq, D, table, caches, kind, rot, axes, inter,
             (cu, torch.tensor(pre, dtype=torch.int32)), positions, axis)


@pytest.mark.parametrize("fmt", list(TYPES))
@pytest.mark.parametrize("rot,inter", [(64, True), (30, False), (40, False)])
def test_append_long_decode_batches(cuda_device, fmt, rot, inter):
    """700 requests of four tokens each, padding among them."""
    B, dql, H, Hq, D, MB = 700, 4, 1, 2, 64, 2
    qkv, table, caches, _, kind = _setup(B * dql, H, Hq, D, B, MB, fmt, rot)
    seq = torch.randint(0, MB * 128 + 1, (B,), generator=torch.Generator().manual_seed(rot), dtype=torch.int32)
    seq[::6] = 0
    _compare(cuda_device, "decode", qkv, H, Hq, D, table, caches, kind, rot, 1, inter, (seq, dql), None, None)
