"""Every 8-bit code as a value of the paged attention.  All tokens hold the same values, so
the output is that value whatever the weights: those are off by less than a quarter of
bf16's half step, and every code is a bf16 number, so it is that number exactly."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_paged_attention import KIND

pytestmark = pytest.mark.gpu

FORMS = [("decode", (1, [1, 5, 128, 129, 700])), ("decode", (3, [400])), ("varlen", [(200, 300), (7, 0), (140, 1000)])]


def _run(dev, fmt, form, rows, D, window, sinks, scale, seed, change=None):
    """[T, H, G, D] outputs with H * D = 256 codes, the codes in order."""
    g = torch.Generator().manual_seed(seed)
    H, G = 256 // D, 5
    dtype = KIND[fmt][0]
    need = max(n if form == "decode" else sum(n) for n in (rows[1] if form == "decode" else rows))
    MB = -(-need // 128)
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 1, H, D).expand(MB * 8, 16, H, D).contiguous()
    if change is not None:
        change(codes)
    k = (torch.randn(codes.shape, generator=g) * 20).to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
    scales = torch.full((MB * 8, H), 1 / 50.0), torch.full((MB * 8, H), scale)
    if form == "decode":
        dql, lens = rows
        T, R, more, fn = dql * len(lens), len(lens), (i32(lens), dql), bsa.bsa_paged_attention_decode
    else:
        T, R, fn = sum(n for n, _ in rows), len(rows), bsa.bsa_paged_attention_varlen
        more = (i32(np.cumsum([0] + [n for n, _ in rows])), i32([p for _, p in rows]))
    table = i32(np.tile(np.arange(MB, dtype=np.int32), (R, 1)))
    q = torch.randn((T, H, G, D), generator=g).to(torch.bfloat16)
    return fn(q.to(dev), k.to(dev), codes.view(dtype).to(dev), table, *more, k_scale=scales[0].to(dev), v_scale=scales[1].to(dev),
              window=window, sinks=sinks).cpu()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("form,rows", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 3)])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -30])
def test_every_code(cuda_device, fmt, form, rows, D, window, sinks, scale):
    got = _run(cuda_device, fmt, form, rows, D, window, sinks, scale, 400 + D)
    want = (torch.arange(256, dtype=torch.int32).to(torch.uint8).view(KIND[fmt][0]).float() * scale).to(torch.bfloat16)
    want = want.view(1, -1, 1, D).expand(got.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(3.0, 4e38, -4e38), want.nan_to_num(3.0, 4e38, -4e38))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("form,rows", FORMS)
@pytest.mark.parametrize("D", [64, 256])
def test_codes_that_are_not_finite_times_zero(cuda_device, fmt, form, rows, D):
    """A scale of zero: zeros, and NaN in the dimensions whose codes are infinite or NaN."""
    got = _run(cuda_device, fmt, form, rows, D, None, 0, 0.0, 410 + D)
    finite = torch.isfinite(torch.arange(256, dtype=torch.int32).to(torch.uint8).view(KIND[fmt][0]).float())
    finite = finite.view(1, -1, 1, D).expand(got.shape)
    assert torch.isnan(got[~finite]).all() and (got[finite] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("form,rows", FORMS)
def test_one_token_that_is_not_finite_among_all_codes(cuda_device, fmt, form, rows):
    """In the third token, whole tiles and partly seen ones: the rows from its position on have it, in its
    dimensions, and infinities of both signs are NaN."""
    D = 128
    odd = {5: 0x7F, 9: 0xFF}
    if fmt == "e5m2":
        odd |= {20: 0x7C, 21: 0xFC, 130: 0x7C}

    def plant(codes):
        codes[..., :] = 0x3C          # 1.5 or 1
        for d, c in odd.items():
            codes[0, 2, d // D, d % D] = c
        if fmt == "e5m2":
            codes[0, 1, 1, 2] = 0xFC  # beside dimension 130's

    got = _run(cuda_device, fmt, form, rows, D, None, 0, 1.0, 420, plant)
    pos = np.concatenate([np.arange(n - rows[0], n) for n in rows[1]] if form == "decode" else [np.arange(p, p + n) for n, p in rows])
    want = torch.full(got.shape, 1.5 if fmt == "e4m3" else 1.0)
    for t, p in enumerate(pos):
        for d, c in odd.items():
            if p >= 2:
                want[t, d // D, :, d % D] = {0x7C: float("inf"), 0xFC: -float("inf")}.get(c, float("nan"))
        if fmt == "e5m2" and p >= 1:
            want[t, 1, :, 2] = -float("inf") if p == 1 else float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.float().nan_to_num(3.0, 4e38, -4e38), want.nan_to_num(3.0, 4e38, -4e38))
