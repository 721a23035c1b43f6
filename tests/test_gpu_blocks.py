"""Forked, grown and freed requests and compacted blocks against the oracle: all
integers and bytes, so everything is equal."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from oracle import blocks

pytestmark = pytest.mark.gpu


class State:
    """A random reachable state of n blocks, and tensors of several shapes and types."""

    def __init__(self, seed, n, MB, dev, R=6, steps=4, tensors=True, most=300):
        rng = np.random.default_rng(seed)
        self.n, self.MB, self.dev, self.rng = n, MB, dev, rng
        rows, lens, refs = [[] for _ in range(R)], [0] * R, [0] * n
        for _ in range(steps):
            parent = rng.integers(-1, len(rows), R).tolist()
            more = rng.integers(0, most, R).tolist()
            (rows, lens, refs), _ = blocks.fork(rows, lens, refs, parent, more, [], MB)
        assert all(b >= 0 for row in rows for b in row)
        # scattered ids
        ids = rng.permutation(n).tolist()
        self.rows, self.lens = [[ids[b] for b in row] for row in rows], lens
        self.refs = [0] * n
        for b, k in enumerate(refs):
            self.refs[ids[b]] = k
        g = torch.Generator().manual_seed(seed)
        self.tensors = [] if not tensors else [
            torch.randint(-2**31, 2**31, (n * 8, 16, 2, 24), generator=g).to(torch.int32).view(torch.bfloat16),
            torch.randint(0, 256, (n * 8, 16, 1, 64), generator=g).to(torch.uint8).view(torch.float8_e4m3fn),
            torch.randn((n * 8, 2), generator=g),
            torch.randn((n, 24), generator=g).to(torch.bfloat16),
            torch.randint(0, 100, (n, 37, 4), generator=g).to(torch.int32),
        ]

    def table(self, rows=None, fill=5):
        t = np.full((len(self.rows if rows is None else rows), self.MB), fill, dtype=np.int32)
        for r, row in enumerate(self.rows if rows is None else rows):
            t[r, :len(row)] = row
        return t

    def on_device(self):
        i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device=self.dev)      # noqa: E731
        return [t.to(self.dev) for t in self.tensors], i32(self.table()), i32(self.lens), i32(self.refs)

    def contents(self):
        return [[b for b in x.view(torch.uint8).reshape(self.n, -1).numpy()] for x in self.tensors]


def same_tensors(tensors, contents):
    for x, c in zip(tensors, contents):
        got = x.cpu().view(torch.uint8).reshape(len(c), -1).numpy()
        assert np.array_equal(got, np.stack(c))


def check_fork(st, parent, more, in_place=False, status=0):
    dev = st.dev
    tensors, table, lens, refs = st.on_device()
    p = torch.tensor(parent, dtype=torch.int32, device=dev)
    m = None if more is None else torch.tensor(more, dtype=torch.int32, device=dev)
    outs = dict(table_out=table, lens_out=lens, refs_out=refs) if in_place else {}
    kept = [x.clone() for x in (table, lens, refs)]
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        got = bsa.bsa_fork_requests(tensors, table, lens, refs, p, m, **outs)
        # a row that would outgrow the table is clamped, and reported
        grown = [(st.lens[q] if q >= 0 else 0) + k for q, k in zip(parent, more or [0] * len(parent))]
        clamped = any(k > st.MB * 128 for k in grown)
        assert bsa.bsa_read_status() == status | (bsa.BSA_STATUS_BAD_CONTEXT if clamped else 0)
    finally:
        bsa.bsa_set_status_word(None)
    contents = st.contents()
    (rows, new_lens, new_refs), short = blocks.fork(st.rows, st.lens, st.refs, parent, more or [0] * len(parent), contents, st.MB)
    assert np.array_equal(got[0].cpu().numpy(), st.table(rows, -1))
    assert got[1].tolist() == new_lens and got[2].tolist() == new_refs
    same_tensors(tensors, contents)
    if in_place:
        assert got[0] is table and got[1] is lens and got[2] is refs
    else:
        assert all(torch.equal(a, b) for a, b in zip(kept, (table, lens, refs)))
    return short


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_fork(cuda_device, seed, in_place):
    st = State(seed, 90, 8, cuda_device)
    rng = np.random.default_rng(100 + seed)
    check_fork(st, rng.integers(-1, 6, 6).tolist(), rng.integers(0, 260, 6).tolist(), in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("parent,more", [
    ([0, 1, 2, 3, 4, 5], None), ([-1] * 6, None), ([5, 4, 3, 2, 1, 0], [1] * 6), ([2] * 6, [0, 1, 127, 128, 129, 0]),
    ([0, 0, 2, 2, -1, -1], [1, 1, 1, 1, 400, 0]),
])
def test_fork_patterns(cuda_device, parent, more, in_place):
    """Nothing, everything freed, a reversal, one parent for all, halves."""
    check_fork(State(11, 90, 8, cuda_device), parent, more, in_place)


@pytest.mark.parametrize("which", [("table",), ("lens",), ("refs",), ("table", "refs"), ("lens", "refs")])
def test_fork_with_some_outputs_in_place(cuda_device, which):
    """Each output in the place of its input by itself: the same state."""
    st = State(18, 90, 8, cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)      # noqa: E731
    parent, more = i32([3, 3, 0, -1, 0, 5]), i32([1, 140, 0, 3, 7, 1])
    tensors, table, lens, refs = st.on_device()
    want = bsa.bsa_fork_requests(tensors, table, lens, refs, parent, more)
    mine, table, lens, refs = st.on_device()
    given = {f"{k}_out": v for k, v in (("table", table), ("lens", lens), ("refs", refs)) if k in which}
    got = bsa.bsa_fork_requests(mine, table, lens, refs, parent, more, **given)
    for a, b in zip((*got, *mine), (*want, *tensors)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(any(g is v for g in got) for v in given.values())


def test_parents_in_one_buffer_with_lengths(cuda_device):
    """Inputs may share memory with each other; a row's parent may be any, several times over."""
    st = State(19, 300, 8, cuda_device)
    tensors, table, lens, refs = st.on_device()
    both = torch.cat([torch.tensor([2, 2, 2, 5, 5, 2], dtype=torch.int32, device=cuda_device), lens % 50])
    got = bsa.bsa_fork_requests(tensors, table, lens, refs, both[:6], both[6:])
    contents = st.contents()
    (rows, new_lens, new_refs), _ = blocks.fork(st.rows, st.lens, st.refs, [2, 2, 2, 5, 5, 2], [n % 50 for n in st.lens],
                                                contents, st.MB)
    assert np.array_equal(got[0].cpu().numpy(), st.table(rows, -1)) and got[1].tolist() == new_lens
    assert got[2].tolist() == new_refs
    same_tensors(tensors, contents)


@pytest.mark.parametrize("rows", [0, 1, 3, 40])
def test_fork_to_another_number_of_rows(cuda_device, rows):
    st = State(12, 200, 8, cuda_device)
    rng = np.random.default_rng(rows)
    check_fork(st, rng.integers(-1, 6, rows).tolist(), rng.integers(0, 150, rows).tolist())


def test_fork_from_nothing_and_without_tensors(cuda_device):
    st = State(13, 50, 5, cuda_device, R=0, steps=0, tensors=False)
    check_fork(st, [-1] * 7, [0, 1, 128, 129, 640, 5, 0])
    st = State(14, 300, 4, cuda_device, tensors=False)
    check_fork(st, [0, 0, 1, 1], [1, 2, 3, 4])


def test_fork_of_many_rows(cuda_device):
    """More rows and blocks than the plan has threads."""
    st = State(15, 40000, 16, cuda_device, R=3000, steps=2, tensors=False, most=900)
    st.tensors = [torch.randint(0, 1000, (st.n, 4), generator=torch.Generator().manual_seed(1)).to(torch.int32)]
    rng = np.random.default_rng(15)
    for in_place in (False, True):
        check_fork(st, rng.integers(-1, 3000, 3000).tolist(), rng.integers(0, 300, 3000).tolist(), in_place)


def test_fork_without_blocks_left(cuda_device):
    """Blocks go out in order; what is left over is -1, its contents lost, and the status says so."""
    st = State(16, 22, 8, cuda_device, R=4, steps=2, most=250)
    assert check_fork(st, [0, 0, 1, 1], [600, 600, 600, 500], status=bsa.BSA_STATUS_NO_BLOCK)


def test_fork_clamps_and_reports(cuda_device):
    dev = cuda_device
    st = State(17, 90, 4, dev, most=120)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        tensors, table, lens, refs = st.on_device()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        for parent, more, same in (([6, 1, 2], [0, 0, 0], ([-1, 1, 2], [0, 0, 0])), ([0, -2, 2], [0, 0, 0], ([0, -1, 2], [0, 0, 0])),
                                   ([0, 1, 2], [-5, 0, 0], ([0, 1, 2], [0, 0, 0])),
                                   ([0, 1, -1], [0, 0, 2**31 - 1], ([0, 1, -1], [0, 0, 512]))):
            got = bsa.bsa_fork_requests(tensors, table, lens, refs, i32(parent), i32(more))
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_CONTEXT
            want = bsa.bsa_fork_requests(tensors, table, lens, refs, i32(same[0]), i32(same[1]))
            assert bsa.bsa_read_status() == 0
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        for n in (-3, 513):
            long = lens.clone()
            long[0] = n
            got = bsa.bsa_fork_requests(tensors, table, long, refs, i32([0]))
            assert bsa.bsa_read_status() & bsa.BSA_STATUS_BAD_CONTEXT
            assert got[1].tolist() == [0 if n < 0 else 512]
        # entries outside the cache are carried on
        bad = table.clone()
        r = max(range(6), key=lambda r: st.lens[r])
        assert st.lens[r] > 128
        bad[r, 0] = st.n
        got = bsa.bsa_fork_requests(tensors, bad, lens, refs, i32([r, r]))
        assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID and got[0][:, 0].tolist() == [st.n] * 2
    finally:
        bsa.bsa_set_status_word(None)


def check_compact(st, in_place=False):
    tensors, table, lens, refs = st.on_device()
    outs = dict(table_out=table, refs_out=refs) if in_place else {}
    got = bsa.bsa_compact_blocks(tensors, table, lens, refs, **outs)
    contents = st.contents()
    before = [list(c) for c in contents]
    rows, new_refs, ids = blocks.compact(st.rows, st.refs, contents)
    assert np.array_equal(got[0].cpu().numpy(), st.table(rows, -1))
    assert got[1].tolist() == new_refs and got[2].tolist() == ids
    same_tensors(tensors, contents)
    del before


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed,n,MB,R", [(1, 90, 8, 6), (2, 300, 8, 6), (3, 61, 4, 1), (4, 1, 1, 1), (5, 9000, 8, 2), (6, 64, 8, 6)])
def test_compact(cuda_device, seed, n, MB, R, in_place):
    check_compact(State(seed, n, MB, cuda_device, R=R, most=100 if n < 60 else 300), in_place)


def test_compact_when_all_or_none_are_in_use(cuda_device):
    st = State(7, 20, 4, cuda_device, R=0, steps=0)
    check_compact(st)
    st.refs = [1] * 20                  # other tables hold them
    check_compact(st)
    st.refs = [0] * 10 + [2] * 10
    check_compact(st)


def test_compact_of_a_large_cache(cuda_device):
    st = State(8, 40000, 16, cuda_device, R=3000, steps=2, tensors=False, most=900)
    st.tensors = [torch.randint(0, 1000, (st.n, 4), generator=torch.Generator().manual_seed(1)).to(torch.int32)]
    for in_place in (False, True):
        check_compact(st, in_place)


def test_compact_reports_entries_without_a_block(cuda_device):
    dev = cuda_device
    st = State(9, 90, 8, dev)
    tensors, table, lens, refs = st.on_device()
    r = max(range(6), key=lambda r: st.lens[r])
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        for entry in (-1, st.n, 2**31 - 1, st.refs.index(0)):
            bad = table.clone()
            bad[r, 0] = entry
            got = bsa.bsa_compact_blocks(tensors, bad, lens, refs)
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID and int(got[0][r, 0]) == -1
            tensors = st.on_device()[0]
        long = lens.clone()
        long[0] = st.MB * 128 + 1
        bsa.bsa_compact_blocks(tensors, table, long, refs)
        assert bsa.bsa_read_status() & bsa.BSA_STATUS_BAD_CONTEXT
    finally:
        bsa.bsa_set_status_word(None)


def test_many_tensors_and_whole_chunks(cuda_device):
    """Caches of many layers in one call; blocks of a chunk's size and around it."""
    dev = cuda_device
    st = State(20, 64, 6, dev)
    g = torch.Generator().manual_seed(20)
    for sizes in ([16, 32768, 32752, 32784, 65536, 98320], [48] * 200):
        st.tensors = [torch.randint(0, 256, (st.n, s), generator=g).to(torch.uint8) for s in sizes]
        check_fork(st, [0, 0, 0, 3, 3, 1], [1, 0, 5, 0, 130, 0])
        check_compact(st)


def test_graph_replays(cuda_device):
    """A step captured in place, replayed: the state moves on as in single calls."""
    dev = cuda_device
    st = State(21, 120, 8, dev, most=100)
    tensors, table, lens, refs = st.on_device()
    parent = torch.tensor([1, 1, 0, 3, 4, 5], dtype=torch.int32, device=dev)
    more = torch.tensor([30, 1, 0, 2, 1, 60], dtype=torch.int32, device=dev)
    start = [x.clone() for x in (table, lens, refs, *tensors)]
    state = [table, lens, refs]

    def step(t, ln, rf, x):
        bsa.bsa_fork_requests(x, t, ln, rf, parent, more, table_out=t, lens_out=ln, refs_out=rf)
        bsa.bsa_compact_blocks(x, t, ln, rf, table_out=t, refs_out=rf, new_ids=ids)

    ids = torch.empty(st.n, dtype=torch.int32, device=dev)
    other = [x.clone() for x in start]
    for _ in range(4):
        step(*other[:3], other[3:])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(*state, tensors)
    for x, s in zip((*state, *tensors), start):
        assert torch.equal(x.view(torch.uint8), s.view(torch.uint8))
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip((*state, *tensors), other))


def test_refusals(cuda_device):
    dev = cuda_device
    st = State(22, 90, 8, dev)
    tensors, table, lens, refs = st.on_device()
    parent = torch.zeros(6, dtype=torch.int32, device=dev)
    fork, compact = bsa.bsa_fork_requests, bsa.bsa_compact_blocks
    n, z = st.n, lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)      # noqa: E731
    for bad in ([tensors[0][:-1]], [tensors[0].transpose(1, 2)], [tensors[0].cpu()], [None], 5, [z(n, 4), z(n * 2, 4)],
                [z(n, 4)[:, :2]]):
        with pytest.raises((ValueError, TypeError)):
            fork(bad, table, lens, refs, parent)
        with pytest.raises((ValueError, TypeError)):
            compact(bad, table, lens, refs)
    for bad in ((table.long(), lens, refs, parent), (table, lens[:-1], refs, parent), (table, lens, refs.cpu(), parent),
                (table, lens, refs, None), (table, lens, refs, parent.float()), (table, lens, refs, parent, z(5))):
        with pytest.raises(ValueError):
            fork(tensors, *bad)
    for kw in (dict(table_out=z(5, 8)), dict(lens_out=z(7)), dict(refs_out=z(n + 1)), dict(workspace=torch.empty(8))):
        with pytest.raises(ValueError):
            fork(tensors, table, lens, refs, parent, **kw)
    both = z(6 + 6)
    shared = z(n, 4)
    for call, status in (
            (lambda: fork([z(n, 3)], table, lens, refs, parent), -7), (lambda: fork([shared, shared], table, lens, refs, parent), -2),
            (lambda: fork(tensors, table, lens, refs, parent, lens_out=parent), -2),
            (lambda: fork(tensors, table, lens, refs, parent, lens_out=both[3:9], new_tokens=both[:6]), -2),
            (lambda: fork(tensors, table, lens, refs, parent, workspace=z(64)), -5),
            (lambda: compact(tensors, table, lens, refs, new_ids=refs), -2),
            (lambda: compact([refs.view(n, 1).expand(n, 1).contiguous()], table, lens, refs), -7),
            (lambda: compact(tensors, table, lens, refs, workspace=z(64)), -5)):
        with pytest.raises(bsa.BsaError) as e:
            call()
        assert e.value.status == status
    with pytest.raises(ValueError):
        fork([shared] * 513, table, lens, refs, parent)
