"""Keys and values that are not finite, for the rows that see them and for the
rows that do not; rows that share a tile with them keep their results."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_paged_attention import KIND, Case, compare

pytestmark = pytest.mark.gpu

NOT_FINITE = {"bf16": [float("nan"), float("inf"), float("-inf")], "e4m3": [float("nan")],
              "e5m2": [float("nan"), float("inf"), float("-inf")]}


def _place(case, b, j):
    return int(case.table[b, j // 128]) * 8 + j % 128 // 16, j % 16


def _expected(case, values):
    """The oracle's result on finite values, and which outputs the planted ones decide:
    {(row, h, d): value}."""
    dev_rows = {}
    for b, j, h, d, v in values:
        for t in np.nonzero((case.req == b) & (case.pos >= j))[0]:
            if case.window and j <= case.pos[t] - case.window and j >= case.sinks:
                continue
            dev_rows.setdefault((int(t), h, d), []).append(v)
    return dev_rows


CASES = [
    ("varlen", (1, [(70, 300), (9, 0), (140, 130)]), 2, 3, 64, 0, 0), ("varlen", (0, [(200, 100)]), 1, 8, 128, 0, 0),
    ("varlen", (0, [(40, 500)]), 1, 2, 256, 0, 0), ("decode", (4, [400, 130, 3]), 2, 4, 128, 0, 0),
    ("decode", (2, [1500]), 1, 8, 64, 0, 0), ("varlen", (0, [(150, 400)]), 1, 4, 128, 90, 20),
    ("decode", (3, [700, 200]), 1, 5, 256, 150, 3),
]


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("form,rows,H,G,D,window,sinks", CASES)
def test_values_that_are_not_finite(cuda_device, fmt, form, rows, H, G, D, window, sinks):
    """Planted in tokens that every row, some rows or (behind a window) no row sees:
    rows that see one have it in that dimension, the others are as without it."""
    case = Case(form, rows, H, G, D, fmt, window, sinks, seed=60 + D)
    rng = np.random.default_rng(61)
    plain = case.c[1].clone()
    planted = []
    for b in np.unique(case.req[case.pos >= 0]):
        last = int(case.pos[case.req == b].max())
        for j in {0, last, max(0, last - 1), last // 2, max(0, last - 130), int(rng.integers(0, last + 1))}:
            h, d = int(rng.integers(0, H)), int(rng.integers(0, D))
            v = float(rng.choice(NOT_FINITE[fmt]))
            page, slot = _place(case, b, j)
            case.c[1][page, slot, h, d] = torch.tensor(v).to(case.dtype)
            plain[page, slot, h, d] = torch.tensor(0.0).to(case.dtype)
            planted.append((int(b), j, h, d, v))
    got = case.run(cuda_device).double().cpu().numpy()
    decided = _expected(case, planted)
    fixed = got.copy()
    for (t, h, d), vs in decided.items():
        want = sum(vs)              # inf - inf and NaN: NaN
        for g in range(G):
            x = got[t, h, g, d]
            assert np.isnan(x) if np.isnan(want) else x == want, (t, h, g, d, x, vs)
        fixed[t, h, :, d] = 0.0
    # everything else, against the same case without them
    case.c[1] = plain
    want = case.want()
    for t, h, d in decided:
        want[t, h, :, d] = 0.0
    mag = case.want(magnitude=True)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 1e-30
    assert np.isfinite(fixed).all()
    assert (np.abs(fixed - want) <= tol).all()


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("form,rows,H,G,D,window,sinks", CASES)
def test_keys_that_are_not_finite(cuda_device, fmt, form, rows, H, G, D, window, sinks):
    """A key of NaN makes the rows that see it NaN, in its KV head, and no others."""
    case = Case(form, rows, H, G, D, fmt, window, sinks, seed=70 + D)
    seen = np.zeros((case.q.shape[0], H), dtype=bool)
    plain = case.c[0].clone()
    for b in np.unique(case.req[case.pos >= 0]):
        last = int(case.pos[case.req == b].max())
        for j in (last, max(0, last - 60)):
            page, slot = _place(case, b, j)
            case.c[0][page, slot, 0, 5] = float("nan")
            plain[page, slot, 0, 5] = 0.0
            rows_ = (case.req == b) & (case.pos >= j)
            if window:
                rows_ &= (j > case.pos - window) | (j < sinks)
            seen[rows_, 0] = True
    got = case.run(cuda_device)
    g = got.double().cpu().numpy()
    assert np.isnan(g[seen]).all()
    # the rows that do not see them are as with a finite key there
    case.c[0] = plain
    finite = torch.from_numpy(np.where(seen[:, :, None, None], case.want(), g))
    compare(case, finite)


def test_queries_that_are_not_finite_or_far_apart(cuda_device):
    """A row of NaN or infinite queries is NaN, its neighbours in the tile are not; queries of
    very different sizes keep their bits."""
    for fmt in KIND:
        case = Case("varlen", (0, [(20, 100)]), 1, 4, 64, fmt, seed=80)
        g = torch.Generator().manual_seed(81)
        case.q = (case.q.float() * torch.exp2(torch.randint(-60, 1, (20, 1, 4, 1), generator=g).float())).to(torch.bfloat16)
        case.q[5] *= torch.exp2(-20 * torch.rand(case.q[5].shape, generator=g))
        case.q[7, 0, 1] = 0
        ok = case.q.clone()
        case.q[3, 0, 2, 7] = float("nan")
        case.q[4, 0, 1, 9] = float("inf")
        got = case.run(cuda_device)
        assert torch.isnan(got[3, 0, 2]).all() and torch.isnan(got[4, 0, 1]).all()
        case.q = ok
        got[3, 0, 2] = torch.from_numpy(case.want()[3, 0, 2]).to(got)
        got[4, 0, 1] = torch.from_numpy(case.want()[4, 0, 1]).to(got)
        compare(case, got)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scales_at_the_ends_of_their_range(cuda_device, fmt):
    """Page scales of 0, 2^-149 and 2^100 beside ordinary ones; the tolerance is of the row's
    own magnitude, so the small ones count where they are alone."""
    case = Case("varlen", (0, [(60, 200), (30, 0)]), 2, 3, 64, fmt, seed=90)
    pages = case.table[1, 0].item() * 8 + torch.arange(8)
    case.s[1][pages] = 2.0 ** -149
    case.s[0][case.table[0, 1].item() * 8 + 2] = 0.0
    case.s[1][case.table[0, 0].item() * 8 + 1] = 0.0
    case.s[1][case.table[0, 1].item() * 8 + 3] = 2.0 ** 100
    got = case.run(cuda_device).double().cpu().numpy()
    want, mag = case.want(), case.want(magnitude=True)
    # outputs below bf16's normal range are off by half of its least step
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 2.0 ** -133
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
