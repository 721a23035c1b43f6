"""Host-side argument checks of the paged attention and of the block operators
(no GPU: nothing here launches a kernel)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_topk_gb300 import build
    build.build()
    import block_sparse_attention_topk_gb300 as m
    m.lib()
    return m


NUL = ctypes.c_void_p(0)
FAR = ctypes.c_void_p(0x10000000)


def _args(bsa, **kw):
    a = bsa.PagedAttentionArgs()
    d = dict(q=0x100000, T=8, H=2, G=4, D=64, out=0x200000, cache_dtype=2, k_cache=0x300000, v_cache=0x400000,
             num_pages=64, k_scale=0x500000, v_scale=0x600000, block_table=0x700000, num_reqs=4, max_blocks=2, window=0,
             sinks=0, scale=1.0, workspace=0, workspace_bytes=0)
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(cache_dtype=1), -4), (dict(cache_dtype=4), -4), (dict(T=-1), -2), (dict(H=0), -2), (dict(G=0), -2),
    (dict(G=65), -2), (dict(D=0), -2), (dict(D=72), -2), (dict(D=272), -2), (dict(num_pages=-1), -2),
    (dict(num_pages=1 << 27), -2), (dict(max_blocks=1 << 24), -2), (dict(max_blocks=-1), -2), (dict(window=-1), -2),
    (dict(sinks=-1), -2), (dict(T=1 << 30), -2), (dict(q=0), -1), (dict(out=0), -1), (dict(block_table=0), -1),
    (dict(k_cache=0), -1), (dict(v_scale=0), -1), (dict(q=0x100008), -7), (dict(out=0x200008), -7), (dict(v_cache=0x400004), -7),
    (dict(out=0x100000), -2), (dict(out=0x300000), -2), (dict(out=0x400000 + 64 * 16 * 2 * 64 - 16), -2), (dict(out=0x500000), -2),
    (dict(out=0x700000), -2), (dict(num_reqs=-1), -2),
])
def test_paged_attention_refusals(bsa, bad, code):
    L = bsa.lib()
    a = _args(bsa, **bad)
    assert L.bsa_paged_attention_decode(a, FAR, 2, NUL) == code
    assert L.bsa_paged_attention_varlen(a, FAR, FAR, NUL) == code


def test_paged_attention_form_refusals(bsa):
    L = bsa.lib()
    assert L.bsa_paged_attention_decode(None, FAR, 2, NUL) == -1
    assert L.bsa_paged_attention_varlen(None, FAR, FAR, NUL) == -1
    assert L.bsa_paged_attention_decode(_args(bsa), FAR, 3, NUL) == -6
    assert L.bsa_paged_attention_decode(_args(bsa), FAR, 0, NUL) == -2
    assert L.bsa_paged_attention_decode(_args(bsa), NUL, 2, NUL) == -1
    assert L.bsa_paged_attention_varlen(_args(bsa), NUL, FAR, NUL) == -1
    assert L.bsa_paged_attention_varlen(_args(bsa), FAR, NUL, NUL) == -1
    assert L.bsa_paged_attention_decode(_args(bsa), ctypes.c_void_p(0x200000), 2, NUL) == -2
    assert L.bsa_paged_attention_varlen(_args(bsa), FAR, ctypes.c_void_p(0x200000), NUL) == -2
    empty = _args(bsa, T=0, num_reqs=0, q=0, out=0, k_cache=0, v_cache=0, num_pages=0)
    assert L.bsa_paged_attention_decode(empty, NUL, 1, NUL) == 0
    assert L.bsa_paged_attention_varlen(empty, NUL, NUL, NUL) == 0


def _blocks(bsa, call, tensors=((0x10000000, 64),), n=None, table=0x100000, lens=0x200000, refs=0x300000, R=4, MB=2, N=64,
            parent=0x400000, more=0, R2=4, o=(0x500000, 0x600000, 0x700000), ws=0x800000, wb=1 << 20):
    L = bsa.lib()
    x = (bsa.BlockTensor * max(1, len(tensors)))(*[bsa.BlockTensor(*t) for t in tensors])
    n = len(tensors) if n is None else n
    p = ctypes.c_void_p
    if call == "fork":
        return L.bsa_fork_requests(x, n, p(table), p(lens), p(refs), R, MB, N, p(parent), p(more), R2, *map(p, o), p(ws), wb, NUL)
    return L.bsa_compact_blocks(x, n, p(table), p(lens), p(refs), R, MB, N, *map(p, o), p(ws), wb, NUL)


@pytest.mark.parametrize("call", ["fork", "compact"])
@pytest.mark.parametrize("bad,code", [
    (dict(R=-1), -2), (dict(MB=-1), -2), (dict(N=-1), -2), (dict(N=1 << 28), -2), (dict(R=1 << 20, MB=1 << 20), -2),
    (dict(n=513), -2), (dict(n=-1), -2), (dict(tensors=((0, 64),)), -1), (dict(tensors=((0x10000000, -16),)), -2),
    (dict(tensors=((0x10000000, 24),)), -7), (dict(tensors=((0x10000008, 64),)), -7), (dict(table=0), -1), (dict(lens=0), -1),
    (dict(refs=0), -1), (dict(o=(0, 0x600000, 0x700000)), -1), (dict(o=(0x500000, 0, 0x700000)), -1),
    (dict(o=(0x500000, 0x600000, 0)), -1), (dict(o=(0x500000, 0x500000, 0x700000)), -2), (dict(o=(0x200000, 0x600000, 0x700000)), -2),
    (dict(o=(0x100004, 0x600000, 0x700000)), -2), (dict(ws=0), -5), (dict(ws=0x800080), -5), (dict(wb=100), -5),
    (dict(tensors=((0x100000, 64),)), -2), (dict(tensors=((0x10000000, 64), (0x10000000 + 4080, 64))), -2),
])
def test_block_refusals(bsa, call, bad, code):
    assert _blocks(bsa, call, **bad) == code


def test_fork_refusals(bsa):
    assert _blocks(bsa, "fork", R2=-1) == -2
    assert _blocks(bsa, "fork", parent=0) == -1
    assert _blocks(bsa, "fork", o=(0x100000, 0x600000, 0x700000), R2=5) == -2          # in place with other rows
    assert _blocks(bsa, "fork", o=(0x500000, 0x200000, 0x700000), R2=5) == -2
    assert _blocks(bsa, "fork", o=(0x500000, 0x400000, 0x700000)) == -2                 # lens_out over parent
    assert _blocks(bsa, "fork", o=(0x500000, 0x600000, 0x400000)) == -2
    assert _blocks(bsa, "compact", o=(0x500000, 0x600000, 0x200000)) == -2              # new_ids over seq_lens
    assert _blocks(bsa, "compact", o=(0x500000, 0x600000, 0x300000)) == -2


def test_workspace_sizes(bsa):
    L = bsa.lib()
    assert L.bsa_fork_workspace_bytes(4, 4, 2, 64) > 0 and L.bsa_fork_workspace_bytes(-1, 4, 2, 64) == 0
    assert L.bsa_compact_workspace_bytes(64) >= 3 * 256 and L.bsa_compact_workspace_bytes(-1) == 0
    # grows with each size
    assert L.bsa_fork_workspace_bytes(4000, 4, 200, 64) > L.bsa_fork_workspace_bytes(4, 4, 200, 64)
    assert L.bsa_fork_workspace_bytes(4, 4000, 200, 64) > L.bsa_fork_workspace_bytes(4, 4, 200, 64)


def test_binding_wants_cuda_tensors(bsa):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)      # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        bsa.bsa_fork_requests([], i(2, 3), i(2), i(9), i(2))
    with pytest.raises(ValueError, match="CUDA"):
        bsa.bsa_compact_blocks([], i(2, 3), i(2), i(9))
    q = torch.zeros((2, 1, 1, 64), dtype=torch.bfloat16)
    c = torch.zeros((8, 16, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bsa.bsa_paged_attention_decode(q, c, c, i(2, 3), i(2), 1)
    with pytest.raises(ValueError):
        bsa.bsa_paged_attention_decode(q, c, c, i(2, 3), i(2), 1, window=0)
    with pytest.raises(TypeError):
        bsa.bsa_paged_attention_decode(q, c, c, i(2, 3), i(2), 1.5)
