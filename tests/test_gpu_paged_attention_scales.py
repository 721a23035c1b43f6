"""Paged attention over an 8-bit cache whose page scales are of no use to a row: scales
of pages that nobody sees, which the append leaves as they were, scales far above the
others in pages that only other rows see, and scales of zero under large scores.

Tolerance as in test_gpu_paged_attention.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged_attention import KIND, Case, check, compare

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "e5m2"]
GARBAGE = [float("nan"), float("inf"), -1.0, 3e38, 2.0 ** -149]
SHAPES = [
    ("decode", (1, [1, 17, 130, 400, 1000, 0]), 2, 8, 128, 0, 0), ("decode", (3, [700, 45, 3, 128]), 1, 4, 64, 0, 0),
    ("decode", (2, [333, 5]), 2, 3, 256, 0, 0), ("varlen", (1, [(70, 300), (9, 0), (140, 130)]), 2, 3, 64, 0, 0),
    ("varlen", (0, [(200, 100), (33, 2)]), 1, 8, 128, 0, 0), ("varlen", (0, [(40, 470)]), 1, 2, 256, 0, 0),
    ("decode", (1, [900, 60, 2000]), 2, 8, 128, 90, 20), ("varlen", (0, [(150, 401), (20, 900)]), 1, 4, 128, 70, 5),
    ("varlen", (0, [(100, 333)]), 1, 4, 256, 50, 0),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form,rows,H,G,D,window,sinks", SHAPES)
def test_scales_of_pages_that_no_row_sees(cuda_device, fmt, form, rows, H, G, D, window, sinks):
    """They are whatever the memory held: not finite, negative, as large or as small as can be."""
    case = Case(form, rows, H, G, D, fmt, window, sinks, seed=200 + D)
    unseen = torch.isnan(case.c[0].float()).flatten(1).all(1)
    assert 8 <= int(unseen.sum()) < unseen.numel()
    g = torch.Generator().manual_seed(201)
    for s in case.s:
        s[unseen] = torch.tensor(GARBAGE)[torch.randint(0, len(GARBAGE), (int(unseen.sum()), H), generator=g)]
    check(case, cuda_device)
    # each kind in all of them
    for x in GARBAGE:
        for s in case.s:
            s[unseen] = x
        check(case, cuda_device)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,D", [(8, 128), (3, 64), (4, 256)])
@pytest.mark.parametrize("large", [2.0 ** 60, 2.0 ** 120])
def test_a_large_scale_behind_a_row(cuda_device, fmt, G, D, large):
    """The prompt's last page has a scale far above the others': the rows before it do not see it."""
    case = Case("varlen", (0, [(120, 200)]), 2, G, D, fmt, seed=210 + D)
    page = int(case.table[0, 2]) * 8 + 3      # tokens 304 to 319
    case.s[1][page] = large
    case.c[1][page] = (case.c[1][page].float() / KIND[fmt][2]).to(case.dtype)
    got = case.run(cuda_device)
    # the rows that see it are another test's
    got[104:] = torch.from_numpy(case.want()[104:]).to(got)
    compare(case, got)
    assert got[:104].abs().max() < 10


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("form,rows,G,D", [("varlen", (0, [(120, 200)]), 8, 128), ("varlen", (0, [(120, 200)]), 3, 256),
                                           ("decode", (4, [320, 203]), 4, 64)])
def test_a_scale_of_no_use_that_a_row_sees(cuda_device, fmt, scale, form, rows, G, D):
    """Scales have to be finite and not negative; of others a row that sees one is NaN, and no other."""
    case = Case(form, rows, 1, G, D, fmt, seed=215 + D)
    page = int(case.table[0, 2]) * 8 + 3      # tokens 304 to 319
    seen = (case.req == 0) & (case.pos >= 304)
    ordinary = case.s[1][page].clone()
    case.s[1][page] = scale
    got = case.run(cuda_device)
    assert torch.isnan(got[seen]).all() and seen.any()
    case.s[1][page] = ordinary
    got[seen] = torch.from_numpy(case.want()[seen]).to(got)
    compare(case, got)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("form,rows,G,D", [("decode", (1, [300, 1000, 90]), 4, 64), ("varlen", (0, [(140, 100), (20, 700)]), 8, 128),
                                           ("decode", (2, [700]), 3, 256)])
@pytest.mark.parametrize("gap", [140.0, 250.0, 500.0])
def test_a_scale_of_zero_under_the_largest_score(cuda_device, fmt, form, rows, G, D, gap):
    """A token whose page's value scale is 0 scores 2^gap times the others: their part is far below bf16's range."""
    case = Case(form, rows, 1, G, D, fmt, seed=220 + D)
    case.q[:] = 0
    case.q[..., :32] = 32.0
    finite = ~torch.isnan(case.c[0].float())
    case.c[0][..., :32] = torch.where(finite[..., :32], 0.0, case.c[0][..., :32].float()).to(case.dtype)
    for b in range(case.table.shape[0]):
        page = int(case.table[b, 0]) * 8 + 1                      # tokens 16 to 31
        case.s[0][page] = gap * np.log(2) / (32 * 32.0 * D ** -0.5 * 32.0)
        case.c[0][page, 5, :, :32] = 32.0
        case.s[1][page] = 0.0
    compare(case, case.run(cuda_device))
