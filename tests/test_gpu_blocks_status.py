"""What forks and compactions report of a state that is not right: nothing stays unsaid
because a request keeps its row, or because the table is empty."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from tests.test_gpu_blocks import State

pytestmark = pytest.mark.gpu


@pytest.fixture
def word(cuda_device):
    w = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    bsa.bsa_set_status_word(w)
    yield w
    bsa.bsa_set_status_word(None)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("entry", [-1, -(2**31), "n", 2**31 - 1])
def test_bad_entries_of_requests_that_keep_their_rows(cuda_device, word, entry, in_place):
    """A grow step: each held entry outside the cache is reported and carried on, wherever it lies."""
    st = State(17, 90, 4, cuda_device, most=120)
    entry = st.n if entry == "n" else entry
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)      # noqa: E731
    seen = 0
    for r in range(6):
        for j in range(-(-st.lens[r] // 128)):
            tensors, table, lens, refs = st.on_device()
            table[r, j] = entry
            outs = dict(table_out=table, lens_out=lens, refs_out=refs) if in_place else {}
            got = bsa.bsa_fork_requests(tensors, table, lens, refs, i32(range(6)), i32([1, 0, 1, 0, 0, 0]), **outs)
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID, (r, j)
            assert int(got[0][r, j]) == entry
            seen += j < st.lens[r] // 128
        # an entry that is not held is nobody's
        tensors, table, lens, refs = st.on_device()
        table[r, -(-st.lens[r] // 128):] = entry
        bsa.bsa_fork_requests(tensors, table, lens, refs, i32(range(6)))
        assert bsa.bsa_read_status() == 0
    assert seen > 0


@pytest.mark.parametrize("R", [1, 7, 3000])
def test_lengths_past_a_table_without_columns(cuda_device, word, R):
    """Requests that hold tokens in a table of no blocks: forks and compactions say so."""
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=cuda_device)      # noqa: E731
    table, refs, parent = z(R, 0), z(20), torch.arange(R, dtype=torch.int32, device=cuda_device)
    last = z(R)
    last[-1] = 5
    for lens, bad in ((z(R), False), (z(R) + 1, True), (z(R) - 1, True), (last, True)):
        want = bsa.BSA_STATUS_BAD_CONTEXT if bad else 0
        out = bsa.bsa_compact_blocks([], table, lens, refs)
        assert bsa.bsa_read_status() == want and out[0].shape == (R, 0) and int(out[1].sum()) == 0
        out = bsa.bsa_fork_requests([], table, lens, refs, parent)
        assert bsa.bsa_read_status() == want and int(out[1].abs().sum()) == 0
