"""The tensors of a fork or a compaction as any iterable: the call holds what the
iteration makes until it is over, whoever else does."""
import gc

import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
from oracle import blocks
from tests.test_gpu_blocks import State

pytestmark = pytest.mark.gpu


def _ways(stack):
    """The layers of one tensor [layers, ...], which alone the caller holds."""
    return {
        "list": lambda: list(stack), "tuple": lambda: tuple(stack), "stacked": lambda: stack, "generator": lambda: (x for x in stack),
        "map": lambda: map(lambda i: stack[i].view(stack.shape[1], -1), range(len(stack))), "iterator": lambda: iter(list(stack)),
        "dict values": lambda: {i: x for i, x in enumerate(stack)}.values(),
    }


@pytest.mark.parametrize("way", ["list", "tuple", "stacked", "generator", "map", "iterator", "dict values"])
def test_layers_of_one_tensor(cuda_device, way):
    st = State(31, 120, 8, cuda_device, tensors=False)
    layers = torch.randint(0, 1000, (5, st.n, 6, 4), generator=torch.Generator().manual_seed(31)).to(torch.int32)
    st.tensors = list(layers)
    _, table, lens, refs = st.on_device()
    stack = layers.to(cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)      # noqa: E731
    parent, more = [3, 3, 0, 0, 5, 1], [1, 140, 0, 3, 7, 1]
    contents = st.contents()
    state, _ = blocks.fork(st.rows, st.lens, st.refs, parent, more, contents, st.MB)
    before = stack._version
    got = bsa.bsa_fork_requests(_ways(stack)[way](), table, lens, refs, i32(parent), i32(more))
    gc.collect()
    after = stack._version
    assert after >= before + len(layers)      # a view's counter is its base's
    assert np.array_equal(got[0].cpu().numpy(), st.table(state[0], -1)) and got[2].tolist() == state[2]
    for x, c in zip(stack.cpu(), contents):
        assert np.array_equal(x.view(torch.uint8).reshape(st.n, -1).numpy(), np.stack(c))
    rows, new_refs, ids = blocks.compact(state[0], state[2], contents)
    got = bsa.bsa_compact_blocks(_ways(stack)[way](), *got)
    assert stack._version >= after + len(layers)
    assert np.array_equal(got[0].cpu().numpy(), st.table(rows, -1)) and got[1].tolist() == new_refs and got[2].tolist() == ids
    for x, c in zip(stack.cpu(), contents):
        assert np.array_equal(x.view(torch.uint8).reshape(st.n, -1).numpy(), np.stack(c))


def test_tensors_that_nothing_else_holds(cuda_device):
    """Storage that only the iteration's tensors own stays until the call is over, call after call."""
    st = State(32, 120, 8, cuda_device, tensors=False)
    _, table, lens, refs = st.on_device()
    parent = torch.tensor([1, 1, 0, 3, 3, 5], dtype=torch.int32, device=cuda_device)
    want = bsa.bsa_fork_requests([], table, lens, refs, parent)
    torch.cuda.synchronize()
    other = torch.full((64, st.n * 16), 7.0, device=cuda_device)
    for _ in range(20):
        got = bsa.bsa_fork_requests((torch.zeros(st.n, 16, device=cuda_device) for _ in range(64)), table, lens, refs, parent)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert (other == 7).all()


def test_what_is_no_iterable_of_tensors(cuda_device):
    st = State(33, 90, 8, cuda_device)
    tensors, table, lens, refs = st.on_device()
    parent = torch.zeros(6, dtype=torch.int32, device=cuda_device)

    def broken():
        yield tensors[0]
        raise KeyError("gone")

    for bad, error in ((5, TypeError), (None, TypeError), ({"k": tensors[0]}, ValueError), ((x.cpu() for x in tensors), ValueError),
                       (tensors[0], ValueError), (broken(), KeyError), ((tensors[2] for _ in range(513)), ValueError)):
        with pytest.raises(error):
            bsa.bsa_fork_requests(bad, table, lens, refs, parent)
    for bad, error in ((5, TypeError), ({"k": tensors[0]}, ValueError), (broken(), KeyError)):
        with pytest.raises(error):
            bsa.bsa_compact_blocks(bad, table, lens, refs)


def test_a_compaction_leaves_its_inputs(cuda_device):
    """The table, lengths and reference counts, where the outputs are new; the lengths always."""
    st = State(34, 300, 8, cuda_device)
    for in_place in (False, True):
        tensors, table, lens, refs = st.on_device()
        kept = [x.clone() for x in (table, lens, refs)]
        versions = [x._version for x in (table, lens, refs)]
        out = bsa.bsa_compact_blocks(tensors, table, lens, refs, **(dict(table_out=table, refs_out=refs) if in_place else {}))
        assert torch.equal(lens, kept[1]) and lens._version == versions[1]
        if in_place:
            assert out[0] is table and out[1] is refs and table._version > versions[0] and refs._version > versions[2]
        else:
            assert torch.equal(table, kept[0]) and torch.equal(refs, kept[2])
            assert [table._version, refs._version] == [versions[0], versions[2]]
            assert not torch.equal(out[0], table) and not torch.equal(out[1], refs)
