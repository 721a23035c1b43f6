"""Paged attention over an 8-bit cache where the weights of a row lie far apart, and how
far its weights are from exact where they do not.

Tolerance of the first: that of test_gpu_paged_attention.py, relative to A = sum_j p_j |v_j|,
with half a step of bf16's subnormals (2^-134) for its absolute slack.  A token whose value
is zero adds nothing to A, however large its weight, so the other tokens' weights have to be
held to their own size.

Tolerance of the last two: weights (a probability times its page's scale) are two bf16 terms,
the second of what the rounding of the first leaves: off by at most 2^-16 of each; exponentials,
and scales through their logarithm, by 2^-16 more.  A score is off by at most
e = D 2^-24 scale |q| |k|, which moves each weight and their sum by as much, and sums over n
tokens by n 2^-24.  bf16 rounds the output by half a step, 2^-8 of it.
|error| <= 2^-8 |out| + (2^-15 + 2 e + 2 n 2^-24) (1 + 2^-8) A."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
from tests.test_gpu_attention_q8_weights import _appended
from tests.test_gpu_paged_attention import KIND, Case

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "e5m2"]


def _tight(got, want, mag, weights=2.0 ** -8 + 2 * 2.0 ** -10):
    got = got.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(want) + weights * (1 + 2.0 ** -8) * mag + 2.0 ** -134
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), ((err / np.maximum(tol, 1e-300)).max(), err.max(), np.abs(want).max())


def _check_appended(dev, cache, q, forms):
    """Rows of requests that all hold the same blocks, in both forms."""
    codes, scales, _, dtype, kind = cache
    cn, sn = [x.numpy() for x in codes], [x.numpy() for x in scales]
    blocks, D = codes[0].shape[0] // 8, q.shape[-1]
    on = [x.to(dev) for x in (codes[0].view(dtype), codes[1].view(dtype))]
    more = dict(zip(("k_scale", "v_scale"), (x.to(dev) for x in scales)))
    for form, rows in forms:
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        if form == "decode":
            dql, lens = rows
            req, pos = oracle.rows_decode(lens, dql)
            T, R, more_rows, fn = len(lens) * dql, len(lens), (i32(lens), dql), bsa.bsa_paged_attention_decode
        else:
            cu, pre = np.cumsum([0] + [n for n, _ in rows]), [p for _, p in rows]
            req, pos = oracle.rows_varlen(cu, pre, int(cu[-1]))
            T, R, more_rows, fn = int(cu[-1]), len(rows), (i32(cu), i32(pre)), bsa.bsa_paged_attention_varlen
        table = np.tile(np.arange(blocks, dtype=np.int32), (R, 1))
        x = q[:T]
        got = fn(x.to(dev), *on, i32(table), *more_rows, **more)
        some = np.unique(np.concatenate([np.arange(min(T, 4)), np.linspace(0, T - 1, 12).astype(int)]))
        want, mag = (oracle.paged_attention(x[some], cn[0], v, kind, *sn, table, req[some], pos[some], D ** -0.5)
                     for v in (cn[1], cn[1] & 0x7F))
        _tight(got[some], want, mag)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,D", [(2, 64), (8, 128), (16, 128), (3, 256)])
@pytest.mark.parametrize("std", [1.0, 0.1, 1e-3, 1e-6, 1e-12])
def test_pages_of_zeros(cuda_device, fmt, G, D, std):
    """Pages whose values are all zero get the scale 1 from the append, far above
    that of pages with small values: alone, eight in a row, and a whole chunk."""
    n, H = 3000, 1
    g = torch.Generator().manual_seed(G + D)
    v = std * torch.randn((n, H, D), generator=g)
    v[160:176] = 0
    v[1024:1152] = 0
    v[1536:2304] = 0
    cache = _appended(cuda_device, fmt, H, D, v, torch.randn((n, H, D), generator=g))
    assert (cache[1][1][[10] + list(range(64, 72)) + list(range(96, 144))] == 1).all()
    q = torch.randn((400, H, G, D), generator=g).to(torch.bfloat16)
    _check_appended(cuda_device, cache, q, [("decode", (1, [n, 1200])), ("varlen", [(150, n - 150), (3, 1197)]), ("varlen", [(200, 90)])])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,D", [(8, 128), (16, 64), (2, 256)])
@pytest.mark.parametrize("std", [1e-25, 1e-31, 1e-34, 1e-37, 1e-39])
def test_tiny_values(cuda_device, fmt, G, D, std):
    """Scales as the append writes them, down to 2^-126: alone, and with whole blocks of zeros before,
    between and behind."""
    n, H = 3000, 1
    g = torch.Generator().manual_seed(G + D)
    keys = torch.randn((n, H, D), generator=g)
    q = torch.randn((320, H, G, D), generator=g).to(torch.bfloat16)
    for first, last in ((0, 0), (0, 768), (768, 1536), (2304, 3000)):
        v = std * torch.randn((n, H, D), generator=g)
        v[first:last] = 0
        cache = _appended(cuda_device, fmt, H, D, v, keys)
        _check_appended(cuda_device, cache, q, [("decode", (2, [n, 2000])), ("varlen", [(300, n - 300)])])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form,rows,G,D,window,sinks", [
    ("decode", (1, [8192, 1000, 300]), 4, 64, 0, 0), ("decode", (2, [3000]), 8, 128, 0, 0), ("decode", (1, [1500, 700]), 1, 256, 0, 0),
    ("varlen", (0, [(150, 900), (30, 2000)]), 8, 128, 0, 0), ("varlen", (0, [(200, 300)]), 3, 256, 0, 0),
    ("decode", (1, [8000, 3000]), 8, 128, 1000, 16), ("varlen", (0, [(140, 2000)]), 4, 64, 300, 16),
])
@pytest.mark.parametrize("gap", [14.0, 18.0, 40.0, 80.0])
def test_a_token_without_value_takes_the_probability(cuda_device, fmt, form, rows, G, D, window, sinks, gap):
    """One token's score is `gap` above the others' and its value is zero (an attention sink): the
    output is made of weights e^-gap of the largest."""
    case = Case(form, rows, 1, G, D, fmt, window, sinks, seed=230 + D)
    case.s = [torch.full_like(x, float(x.median())) for x in case.s]
    case.q[:] = 0
    case.q[..., :32] = 32.0
    # the first 32 dimensions of the keys alone count: 0, and `gap` in all at the sink
    finite = ~torch.isnan(case.c[0].float())
    case.c[0][..., :32] = torch.where(finite[..., :32], 0.0, case.c[0][..., :32].float()).to(case.dtype)
    unit = gap / (32 * 32.0 * D ** -0.5 * float(case.s[0][0, 0]))
    assert unit < KIND[fmt][2]
    for b in range(case.table.shape[0]):
        page = int(case.table[b, 0]) * 8
        case.c[0][page, 5, :, :32] = unit
        case.c[1][page, 5] = 0
    _tight(case.run(cuda_device), case.want(), case.want(magnitude=True))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gap", [14.0, 40.0, 80.0, 100.0, 150.0, 280.0])
@pytest.mark.parametrize("form,rows,G,D", [("decode", (1, [3000, 500]), 8, 128), ("varlen", (0, [(200, 700)]), 4, 64),
                                           ("decode", (1, [1500]), 2, 256)])
def test_a_page_without_value_takes_the_probability(cuda_device, fmt, form, rows, G, D, gap):
    """The same with the sink in a page whose value scale is zero, the other pages' scales large, so
    that the output is an ordinary number, or one of bf16's smallest, however far the scores are apart."""
    case = Case(form, rows, 1, G, D, fmt, seed=240 + D)
    case.q[:] = 0
    case.q[..., :32] = 32.0
    finite = ~torch.isnan(case.c[0].float())
    case.c[0][..., :32] = torch.where(finite[..., :32], 0.0, case.c[0][..., :32].float()).to(case.dtype)
    case.s[1] *= 2.0 ** 100
    for b in range(case.table.shape[0]):
        page = int(case.table[b, 0]) * 8 + 1
        case.s[0][page] = gap / (32 * 32.0 * D ** -0.5 * 32.0)
        case.c[0][page, 5, :, :32] = 32.0
        case.s[1][page] = 0.0
    _tight(case.run(cuda_device), case.want(), case.want(magnitude=True))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,D", [(8, 128), (3, 64), (4, 256)])
@pytest.mark.parametrize("large", [2.0 ** 20, 2.0 ** 60, 2.0 ** 120])
def test_a_page_with_a_large_scale(cuda_device, fmt, G, D, large):
    """The prompt's last page has a scale far above the others' and values of every size, zeros among
    them: where those are, the outputs of the rows that see it are of the other pages."""
    case = Case("varlen", (0, [(120, 200)]), 2, G, D, fmt, seed=245 + D)
    page = int(case.table[0, 2]) * 8 + 3      # tokens 304 to 319
    case.s[1][page] = large
    case.c[1][page] = (case.c[1][page].float() / KIND[fmt][2]).to(case.dtype)
    case.c[1][page, :, :, ::3] = 0
    got = case.run(cuda_device)
    _tight(got, case.want(), case.want(magnitude=True))
    assert got[104:, ..., ::3].abs().max() < 10 and got[104:].abs().max() > large / 2 ** 14


def _score_error(case):
    """e of the tolerance, for the largest rows."""
    D = case.q.shape[-1]
    k = case.c[0].double().nan_to_num() * case.s[0].double()[:, None, :, None]
    return D * 2.0 ** -24 * D ** -0.5 * float(case.q.double().norm(dim=-1).max()) * float(k.norm(dim=-1).max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form,rows,H,G,D,window,sinks", [
    ("decode", (1, [1, 17, 400, 1000, 3000]), 2, 8, 128, 0, 0), ("decode", (4, [700, 45, 1300]), 2, 4, 64, 0, 0),
    ("varlen", (0, [(200, 1000), (33, 20)]), 1, 8, 128, 0, 0), ("varlen", (0, [(300, 500)]), 2, 3, 64, 0, 0),
    ("varlen", (0, [(40, 900)]), 1, 2, 256, 0, 0), ("decode", (1, [2000, 900]), 2, 5, 256, 0, 0),
    ("decode", (1, [2000, 900, 30]), 2, 8, 128, 500, 4), ("decode", (2, [1000, 300]), 1, 4, 64, 100, 0),
    ("varlen", (0, [(150, 600), (90, 0)]), 2, 4, 128, 200, 10), ("varlen", (0, [(130, 400)]), 1, 6, 64, 77, 0),
    ("varlen", (0, [(60, 700)]), 1, 4, 256, 333, 64),
])
def test_weights_keep_their_bits(cuda_device, fmt, form, rows, H, G, D, window, sinks):
    case = Case(form, rows, H, G, D, fmt, window, sinks, seed=250 + D)
    n = int(case.pos.max()) + 1
    weights = 2.0 ** -15 + 2 * _score_error(case) + 2 * n * 2.0 ** -24
    assert weights < 2.0 ** -9
    _tight(case.run(cuda_device), case.want(), case.want(magnitude=True), weights)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form,rows,G,D", [("decode", (1, [1024] * 8), 8, 128), ("varlen", (0, [(64, 1024)]), 8, 64),
                                           ("varlen", (0, [(70, 700)]), 4, 256)])
def test_error_is_that_of_rounding_the_output(cuda_device, fmt, form, rows, G, D):
    """Over many outputs the error's norm is that of rounding the exact ones to bf16 (2^-8 / sqrt(12)
    and more of each): weights within 2^-15 and scores within 2^-12 add their squares, less than 1 % of it."""
    case = Case(form, rows, 1, G, D, fmt, seed=260 + D)
    want = case.want()
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    own = np.linalg.norm(rounded - want)
    assert np.linalg.norm(case.run(cuda_device).double().cpu().numpy() - want) <= 1.01 * own
