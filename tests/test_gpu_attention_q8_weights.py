"""8-bit attention where the weights p_j vs_j of a row lie far apart, against the
64-bit oracle.

Tolerance: that of tests/test_gpu_attention_q8.py, relative to A = sum_j p_j |v_j|.
A token whose value is zero adds nothing to A, however large its weight, so the
other tokens' weights have to be held to their own size."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
from tests.test_gpu_attention_q8 import KIND, _bound, _case, _check

pytestmark = pytest.mark.gpu


def _appended(dev, fmt, H, D, values, keys):
    """One request's tokens [n, H, D] appended to a fresh cache in table order."""
    dtype, kind, _ = KIND[fmt]
    n = values.shape[0]
    blocks = -(-n // 128)
    kc, vc = (torch.zeros((blocks * 8, 16, H, D), dtype=dtype, device=dev) for _ in range(2))
    ks, vs = (torch.ones((blocks * 8, H), device=dev) for _ in range(2))
    table = torch.arange(blocks, dtype=torch.int32, device=dev)[None]
    bsa.bsa_append_kv_decode(keys.to(torch.bfloat16).to(dev), values.to(torch.bfloat16).to(dev), kc, vc, table,
                             torch.tensor([n], dtype=torch.int32, device=dev), n, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    codes = [x.view(torch.uint8).cpu() for x in (kc, vc)]
    pages = torch.arange(blocks * 8, dtype=torch.int32)
    return codes, [ks.cpu(), vs.cpu()], pages, dtype, kind


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("G,D", [(2, 64), (8, 128), (16, 128), (3, 256)])
@pytest.mark.parametrize("std", [1.0, 0.1, 1e-3, 1e-6, 1e-12])
def test_attention_q8_pages_of_zeros(cuda_device, fmt, G, D, std):
    """Pages whose values are all zero get the scale 1 from the append, far above
    that of pages with small values: alone, eight in a row, and a whole chunk."""
    n, H = 3000, 1
    g = torch.Generator().manual_seed(G + D)
    v = std * torch.randn((n, H, D), generator=g)
    v[160:176] = 0
    v[1024:1152] = 0
    v[1536:2304] = 0
    codes, scales, pages, dtype, kind = _appended(cuda_device, fmt, H, D, v, torch.randn((n, H, D), generator=g))
    assert (scales[1][[10] + list(range(64, 72)) + list(range(96, 144))] == 1).all()
    q = torch.randn((2, H, G, D), generator=g).to(torch.bfloat16)
    bt = pages.expand(2, H, -1).contiguous()
    ctx = torch.tensor([[n], [1200]], dtype=torch.int32)
    _check(cuda_device, q, codes, scales, bt, ctx, dtype, kind)


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("G,D", [(4, 64), (8, 128), (12, 64), (1, 256)])
def test_attention_q8_a_token_without_value_takes_the_probability(cuda_device, fmt, G, D):
    """One token's score is 14 above the others' and its value is zero (an
    attention sink): the output is made of weights 2^-20 of the largest."""
    T, H, K = 2, 1, 12
    q, c, s, bt, ctx, dtype, kind = _case(T, H, G, D, K, fmt, [K * 128, 1000], 3 * G + D)
    s = [torch.full_like(x, float(x.median())) for x in s]
    q[:] = 0
    q[..., :32] = 4.0
    # the first 32 dimensions of the keys alone count: 0, and 14 in all at the sink
    c[0][bt[:, 0].long(), :, 0, :32] = 0
    unit = torch.tensor(14 / (32 * 4.0 * D ** -0.5 * float(s[0][0, 0])))
    assert unit < KIND[fmt][2]
    for t, j in ((0, 5), (1, 700)):
        page = int(bt[t, 0, j // 16])
        c[0][page, j % 16, 0, :32] = unit.to(dtype).view(torch.uint8)
        c[1][page, j % 16, 0] = 0
    _check(cuda_device, q, c, s, bt, ctx, dtype, kind)


def test_attention_q8_error_is_that_of_rounding_the_output(cuda_device):
    """Over many outputs the error's norm is that of rounding the exact ones to
    bf16 (2^-8 / sqrt(12) and more of each): probabilities within 2^-12 and scores
    within 2^-14 add their squares, less than 1 % of it."""
    q, c, s, bt, ctx, dtype, kind = _case(8, 1, 8, 128, 8, "e4m3", [1024] * 8, 77)
    want = oracle.sparse_decode_attention_q8(q, c[0].numpy(), c[1].numpy(), kind, s[0].numpy(), s[1].numpy(),
                                             bt.numpy(), ctx.numpy(), 128 ** -0.5)
    got = bsa.bsa_sparse_decode_attention_q8(
        *(x.to(cuda_device) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)))
    torch.cuda.synchronize()
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    own = np.linalg.norm(rounded - want)
    assert np.linalg.norm(got.double().cpu().numpy() - want) <= 1.01 * own


def _check_small(dev, q, codes, scales, bt, ctx, dtype, kind):
    """_check without its absolute slack: half a step of bf16's subnormals."""
    cn, sn = [x.numpy() for x in codes], [x.numpy() for x in scales]
    sc = q.shape[-1] ** -0.5
    want = oracle.sparse_decode_attention_q8(q, cn[0], cn[1], kind, sn[0], sn[1], bt.numpy(), ctx.numpy(), sc)
    got = bsa.bsa_sparse_decode_attention_q8(*(x.to(dev) for x in (q, codes[0].view(dtype), codes[1].view(dtype),
                                                                   scales[0], scales[1], bt, ctx)))
    torch.cuda.synchronize()
    tol = _bound(q, cn, sn, bt.numpy(), ctx.numpy(), kind, sc, want) - 1e-30 + 2.0 ** -134
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err.max(), np.abs(want).max())


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("T,G,D", [(2, 8, 128), (1, 16, 64), (400, 2, 256)])
@pytest.mark.parametrize("std", [1e-28, 1e-31, 1e-34, 1e-37, 1e-39])
def test_attention_q8_tiny_values(cuda_device, fmt, T, G, D, std):
    """Scales as the append writes them, down to 2^-126: whole rows of tiny values,
    in one CTA and joined, and rows with tiny values beside ordinary ones."""
    n, H = 1300, 1
    g = torch.Generator().manual_seed(G + D)
    v = std * torch.randn((n, H, D), generator=g)
    keys = torch.randn((n, H, D), generator=g)
    q = torch.randn((T, H, G, D), generator=g).to(torch.bfloat16)
    for ordinary in (0, 5):
        v[600:600 + ordinary] = torch.randn((ordinary, H, D), generator=g)
        codes, scales, pages, dtype, kind = _appended(cuda_device, fmt, H, D, v, keys)
        assert scales[1].min() <= 4.5 * std / 8 or scales[1].min() == 2.0 ** -126
        bt = pages.expand(T, H, -1).contiguous()
        ctx = (torch.arange(T, dtype=torch.int32) % 7 * -100 + n).view(T, H)
        _check_small(cuda_device, q, codes, scales, bt, ctx, dtype, kind)


def test_attention_q8_scales_of_zero_and_subnormal_scales(cuda_device):
    """A page whose value scale is 0 or subnormal counts for its probability."""
    q, c, s, bt, ctx, dtype, kind = _case(3, 1, 4, 128, 4, "e4m3", [512, 300, 64], 12)
    s[1][bt[0, 0, 3]] = 0
    s[1][bt[1, 0, ::2].long()] = 2.0 ** -140
    s[1][bt[2, 0, :4].long()] = 0
    _check_small(cuda_device, q, c, s, bt, ctx, dtype, kind)


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("G,D", [(8, 128), (16, 64), (2, 256)])
@pytest.mark.parametrize("std", [1e-25, 1e-31, 1e-34, 1e-37])
def test_attention_q8_tiny_values_beside_blocks_of_zeros(cuda_device, fmt, G, D, std):
    """Whole chunks of zeros, with the scale 1, before, between and behind tokens with
    tiny values, in rows that one CTA walks."""
    n, H, T = 3000, 1, 320
    g = torch.Generator().manual_seed(G + D)
    keys = torch.randn((n, H, D), generator=g)
    q = torch.randn((T, H, G, D), generator=g).to(torch.bfloat16)
    assert bsa.bsa_attention_q8_workspace_bytes(T, H, G, D, 24) == 0
    for first, last in ((0, 768), (768, 1536), (2304, 3000)):
        v = std * torch.randn((n, H, D), generator=g)
        v[first:last] = 0
        codes, scales, pages, dtype, kind = _appended(cuda_device, fmt, H, D, v, keys)
        bt = pages.expand(T, H, -1).contiguous()
        rows = [0, 1, 317]
        ctx = torch.full((T, H), n, dtype=torch.int32)
        got = bsa.bsa_sparse_decode_attention_q8(*(x.to(cuda_device) for x in (
            q, codes[0].view(dtype), codes[1].view(dtype), scales[0], scales[1], bt, ctx)))
        torch.cuda.synchronize()
        cn, sn, sc = [x.numpy() for x in codes], [x.numpy() for x in scales], D ** -0.5
        sub = (q[rows], cn, sn, bt[rows].numpy(), ctx[rows].numpy(), kind, sc)
        want = oracle.sparse_decode_attention_q8(sub[0], cn[0], cn[1], kind, sn[0], sn[1], sub[3], sub[4], sc)
        tol = _bound(*sub, want) - 1e-30 + 2.0 ** -134
        err = np.abs(got[rows].double().cpu().numpy() - want)
        assert (err <= tol).all(), (err.max(), np.abs(want).max())
