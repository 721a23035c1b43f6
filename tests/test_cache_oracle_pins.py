"""Pins of the oracle's rotary, append and 8-bit attention functions (CPU)."""
import math

import numpy as np
import pytest
import torch

import oracle

KINDS = {oracle.E4M3: torch.float8_e4m3fn, oracle.E5M2: torch.float8_e5m2}


@pytest.mark.parametrize("kind", list(KINDS))
def test_code_values_and_rounding(kind):
    """Every code has torch's value; midpoints go to the even code; the range
    saturates; NaN stays NaN."""
    vals = oracle.code_values(kind)
    want = torch.arange(256, dtype=torch.uint8).view(KINDS[kind]).double().numpy()
    assert np.array_equal(vals, want, equal_nan=True)
    fin = np.array([v for v in vals[:128] if np.isfinite(v)])
    mid = (fin[:-1] + fin[1:]) / 2
    got = oracle.codes_of(mid, kind)
    assert (got % 2 == 0).all() and np.array_equal(vals[got], np.where(np.arange(len(mid)) % 2, fin[1:], fin[:-1]))
    assert np.array_equal(oracle.codes_of(np.nextafter(mid, 1e9), kind), np.arange(1, len(fin)))
    top = fin[-1]
    assert np.array_equal(vals[oracle.codes_of([1e9, -1e9, np.inf, -np.inf], kind)], [top, -top, top, -top])
    assert np.isnan(vals[oracle.codes_of([np.nan], kind)]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_complex_product_and_inverts(interleaved):
    rng = np.random.default_rng(1)
    T, H, D, rot = 7, 3, 24, 20
    x = rng.standard_normal((T, H, D))
    pos = rng.integers(0, 1 << 20, (3, T))
    f = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    axis = rng.integers(0, 3, rot // 2)
    y = oracle.rope(x, pos, f, axis, interleaved)
    ang = pos[axis].T * f.astype(np.float64)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * ang)[:, None]
    want = x.copy()
    want[..., a], want[..., b] = z.real, z.imag
    assert np.abs(y - want).max() < 1e-12
    assert np.abs(oracle.rope(y, pos, f, axis, interleaved, inverse=True) - x).max() < 1e-12


def test_append_scales_and_requantisation():
    """A page that fills in two steps: the scale is the smallest power of two
    that holds the page, kept codes follow it, fresh pages forget theirs."""
    H, D = 1, 16
    table = np.array([[1]])
    cache = np.zeros((16, 16, H, D))
    scales = np.full((16, H), 7.0, np.float32)
    x = np.full((3, H, D), 3.0)
    x[1] = 448 * 2.0 ** -5
    c, s, fresh = oracle.append(x, [0, 0, 0], [0, 1, 2], table, oracle.E4M3, cache, scales)
    assert s[8, 0] == 2.0 ** -5 and (s[:8] == 7).all() and fresh[8, :3].all() and fresh.sum() == 3
    assert (c[8, 0] == 96).all() and (c[8, 1] == 448).all()
    y = np.full((1, H, D), 100.0)
    c2, s2, _ = oracle.append(y, [0], [3], table, oracle.E4M3, c, s)
    assert s2[8, 0] == 0.25 and (c2[8, 0] == 12).all() and (c2[8, 1] == 56).all() and (c2[8, 3] == 400).all()
    c3, s3, _ = oracle.append(np.zeros((1, H, D)), [0], [0], table, oracle.E4M3, c2, s2)
    assert s3[8, 0] == 1 and (c3[8, 0] == 0).all() and (c3[8, 1] == 56).all()


def test_append_skips_what_has_no_place():
    cache = np.zeros((8, 16, 1, 16))
    s = np.ones((8, 1), np.float32)
    x = np.ones((4, 1, 16))
    for req, pos, table in (([0] * 4, [-1] * 4, [[0]]), ([0] * 4, [128, 129, 130, 131], [[0]]),
                            ([0] * 4, [0, 1, 2, 3], [[-1]]), ([0] * 4, [0, 1, 2, 3], [[1]])):
        c, _, fresh = oracle.append(x, req, pos, np.array(table), oracle.E4M3, cache, s)
        assert not fresh.any() and not c.any()


@pytest.mark.parametrize("kind", list(KINDS))
def test_attention_q8_against_numpy(kind):
    rng = np.random.default_rng(5)
    T, H, G, D, K, P = 3, 2, 3, 64, 2, 20
    vals = oracle.code_values(kind)
    lim = 120 if kind == oracle.E4M3 else 100
    kc, vc = rng.integers(0, lim, (2, P, 16, H, D), dtype=np.uint8)
    kc[rng.random(kc.shape) < 0.5] |= 0x80
    ks, vs = np.exp2(rng.integers(-10, -6, (2, P, H)).astype(np.float32))
    bt = rng.integers(0, P, (T, H, K * 8)).astype(np.int32)
    ctx = np.array([[0, 1], [17, 130], [256, 999]], np.int32)
    bt[2, 0, 3] = -1
    bt[2, 0, 4] = P
    q = torch.randn((T, H, G, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    got = oracle.sparse_decode_attention_q8(q, kc, vc, kind, ks, vs, bt, ctx, 0.3)
    for t in range(T):
        for h in range(H):
            n = min(int(ctx[t, h]), K * 128)
            j = np.arange(n)
            pg = bt[t, h, j // 16]
            ok = (pg >= 0) & (pg < P)
            pg, j = pg[ok], j[ok]
            k = vals[kc[pg, j % 16, h]] * ks[pg, h][:, None]
            v = vals[vc[pg, j % 16, h]] * vs[pg, h][:, None]
            s = q[t, h].double().numpy() @ k.T * 0.3
            if n == 0:
                assert (got[t, h] == 0).all()
                continue
            p = np.exp(s - s.max(1, keepdims=True))
            want = p @ v / p.sum(1, keepdims=True)
            assert np.abs(got[t, h] - want).max() <= 1e-9 * np.abs(v).max()
    assert math.isclose(float(np.abs(got[0, 1] - vals[vc[bt[0, 1, 0], 0, 1]] * vs[bt[0, 1, 0], 1]).max()), 0, abs_tol=1e-12)
