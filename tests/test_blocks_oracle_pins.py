"""Pins of the oracle's paged attention and of its block states (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import blocks


def test_fork_worked_example():
    """Three requests of 300, 128 and 10 tokens; 0 forks in two, 1 is freed, 2 grows
    past its block; blocks 1 (freed) and 5, 7 (free) are taken in order."""
    rows, lens = [[0, 2, 3], [1], [4]], [300, 128, 10]
    refs = [1, 1, 1, 1, 1, 0, 1, 0]                    # block 6 belongs to another table
    contents = [[10 * b for b in range(8)]]
    (r, n, k), short = blocks.fork(rows, lens, refs, [0, 0, 2], [1, 0, 120], contents, 4)
    assert r == [[0, 2, 3], [0, 2, 1], [4, 5]] and n == [301, 300, 130] and not short
    assert k == [2, 1, 2, 1, 1, 1, 1, 0]
    assert contents == [[0, 30, 20, 30, 40, 50, 60, 70]]
    (r, n, k), short = blocks.fork(r, n, k, [-1, 1, 1, 1], [513, 0, 0, 0], contents, 4)
    assert n == [512, 300, 300, 300] and short and r[0] == [3, 4, 5, 7] and r[1] == [0, 2, 1]
    assert r[2] == [0, 2, -1] and r[3] == [0, 2, -1] and k == [3, 1, 3, 1, 1, 1, 1, 1]


def test_compact_worked_example():
    rows, refs = [[5, 0], [5, 3]], [1, 0, 0, 1, 0, 2, 0]
    contents = [list("abcdefg")]
    r, k, ids = blocks.compact(rows, refs, contents)
    assert ids == [0, -1, -1, 1, -1, 2, -1] and r == [[2, 0], [2, 1]] and k == [1, 1, 2, 0, 0, 0, 0]
    assert contents[0][:3] == ["a", "d", "f"]


@pytest.mark.parametrize("seed", range(8))
def test_states_keep_their_tokens(seed):
    """Random steps: what a row's blocks hold is its parent's content, block by block;
    references count the holders; compaction changes no row's content."""
    rng = np.random.default_rng(seed)
    n, MB = 60, 6
    rows, lens, refs, contents = [[] for _ in range(5)], [0] * 5, [0] * n, [[0] * n]
    stamp = 0
    for step in range(12):
        parent = rng.integers(-1, len(rows), rng.integers(1, 7)).tolist()
        more = rng.integers(0, 200, len(parent)).tolist()
        seen = [[contents[0][b] for b in row] for row in rows]
        (new, new_lens, refs), short = blocks.fork(rows, lens, refs, parent, more, contents, MB)
        assert not short
        for r, p in enumerate(parent):
            old = seen[p] if p >= 0 else []
            assert [contents[0][b] for b in new[r][:len(old)]] == old
            assert new_lens[r] == min((lens[p] if p >= 0 else 0) + more[r], MB * 128)
            assert len(new[r]) == -(-new_lens[r] // 128)
        flat = [b for row in new for b in row]
        assert refs == [flat.count(b) for b in range(n)]
        last = [row[-1] for row, m in zip(new, new_lens) if m % 128]
        assert all(refs[b] == 1 for b in last)
        for row, old in zip(new, [seen[p] if p >= 0 else [] for p in parent]):
            for b in row[len(old):]:
                stamp += 1
                contents[0][b] = stamp
        rows, lens = new, new_lens
        if step % 3 == 2:
            had = [[contents[0][b] for b in row] for row in rows]
            rows, refs, _ = blocks.compact(rows, refs, contents)
            assert [[contents[0][b] for b in row] for row in rows] == had
            assert all(k > 0 for k in refs[:sum(k > 0 for k in refs)])


@pytest.mark.parametrize("kind", [0, oracle.E4M3, oracle.E5M2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3), (130, 200), (1000, 0)])
def test_paged_attention_against_numpy(kind, window, sinks):
    rng = np.random.default_rng(kind * 10 + window)
    H, G, D, MB, pages = 2, 3, 16, 3, 60
    cu, pre, T = [1, 4, 4, 11], [0, 9, 290], 12
    req, pos = oracle.rows_varlen(cu, pre, T)
    table = np.array([[6, 1, 2], [0, 3, 4], [5, 7, -1]])          # 7: half of its pages outside the cache
    table[2, 2] = 3
    x = torch.randn((2, pages, 16, H, D), generator=torch.Generator().manual_seed(window))
    ks, vs = np.exp2(rng.integers(-3, 3, (2, pages, H)).astype(np.float32))
    if kind == 0:
        k, v = (y.to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16) for y in x)
        kv, vv = (y.to(torch.bfloat16).double().numpy() for y in x)
    else:
        dt = torch.float8_e4m3fn if kind == oracle.E4M3 else torch.float8_e5m2
        k, v = (y.to(dt).view(torch.uint8).numpy() for y in x)
        kv, vv = (y.to(dt).double().numpy() * s[:, None, :, None] for y, s in zip(x, (ks, vs)))
    q = torch.randn((T, H, G, D), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    got = oracle.paged_attention(q, k, v, kind, ks, vs, table, req, pos, 0.3, window, sinks)
    for t in range(T):
        j = np.arange(pos[t] + 1)
        if window:
            j = j[(j > pos[t] - window) | (j < sinks)]
        page = table[req[t], j // 128] * 8 + j % 128 // 16
        j, page = j[page < pages], page[page < pages]
        for h in range(H):
            if j.size == 0:
                assert (got[t, h] == 0).all()
                continue
            s = q[t, h].double().numpy() @ kv[page, j % 16, h].T * 0.3
            w = np.exp(s - s.max(1, keepdims=True))
            assert np.abs(got[t, h] - w @ vv[page, j % 16, h] / w.sum(1, keepdims=True)).max() <= 1e-12 * np.abs(vv).max()
    one = oracle.paged_attention(q, k, v, kind, ks, vs, table, req, pos, 0.3, 1, 0)
    assert np.allclose(one[3, 1], vv[table[0, 0] * 8, 2, 1])      # a window of one: the row's own value
