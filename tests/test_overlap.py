"""Calls whose outputs share memory with their inputs are refused (no GPU: CPU
tensors stand in for device tensors in the binding, whose accepted calls end at the
check for a GPU; made-up addresses in the C calls, all of them refused)."""
import ctypes
import random

import pytest
import torch

from tests.test_cache_abi import NUL, P16, _args, _attend, _rope, bsa  # noqa: F401


def _at(x):
    return ctypes.c_void_p(x)


def _memory(t):
    """The element offsets of a 3D view."""
    return {t.storage_offset() + i * t.stride(0) + j * t.stride(1) + k
            for i in range(t.shape[0]) for j in range(t.shape[1]) for k in range(t.shape[2])}


def test_rope_out_beside_x_in_one_buffer(bsa):  # noqa: F811
    pos, inv = torch.zeros(6, dtype=torch.int32), torch.zeros(8)
    buf = torch.zeros((6, 9, 16), dtype=torch.bfloat16)
    rope = lambda x, out: bsa.bsa_rope(x, pos, inv, out=out)  # noqa: E731
    for x, out in ((buf[:, 1:4], buf[:, :3]), (buf[:, :3], buf[:, 2:5]), (buf[:, :3, :], buf.flatten()[8:].as_strided((6, 3, 16), (144, 16, 1), 8)),
                   (buf[:, :3], buf.view(54, 16)[:18].view(6, 3, 16))):
        with pytest.raises(ValueError, match="overlap"):
            rope(x, out)
    for x, out in ((buf[:, :3], buf[:, 3:6]), (buf[:, 6:], buf[:, :3]), (buf[:, :3], buf[:, :3]), (buf[:, ::3], buf[:, 1::3]),
                   (buf[:, :3], torch.zeros((6, 3, 16), dtype=torch.bfloat16)), (buf[:, :1].expand(6, 3, 16), buf[:, 3:6])):
        with pytest.raises(ValueError, match="CUDA device"):
            rope(x, out)


def test_rope_random_views(bsa):  # noqa: F811
    rng = random.Random(3)
    buf = torch.zeros(400)
    seen = set()
    for _ in range(2000):
        T, H, D = rng.randint(1, 4), rng.randint(1, 4), rng.choice((2, 4, 6))
        x, out = (buf.as_strided((T, H, D), (rng.randint(0, 30), rng.randint(0, 30), 1), rng.randint(0, 100)) for _ in range(2))
        if rng.random() < 0.5:
            out = buf.as_strided((T, H, D), x.stride(), rng.randint(0, 100))
        shared = bool(_memory(x) & _memory(out))
        same = x.data_ptr() == out.data_ptr() and (T == 1 or x.stride(0) == out.stride(0)) and (H == 1 or x.stride(1) == out.stride(1))
        seen.add((shared, same))
        with pytest.raises(ValueError, match="overlap" if shared and not same else "CUDA device"):
            bsa.bsa_rope(x, torch.zeros(T, dtype=torch.int32), torch.zeros(1), out=out)
    assert len(seen) == 3


def test_append_outputs_apart(bsa):  # noqa: F811
    T, H, Hq, D, pages = 6, 2, 8, 64, 24
    fused = torch.zeros((T, Hq + 2 * H, D), dtype=torch.bfloat16)
    q, k, v = fused.split([Hq, H, H], dim=1)
    f8 = torch.float8_e4m3fn
    good = dict(k=k, v=v, q=q, k_cache=torch.zeros((pages, 16, H, D), dtype=f8), v_cache=torch.zeros((pages, 16, H, D), dtype=f8),
                block_table=torch.zeros((3, 1), dtype=torch.int32), seq_lens=torch.zeros(3, dtype=torch.int32), decode_query_len=2,
                k_scale=torch.zeros((pages, H)), v_scale=torch.zeros((pages, H)))
    both = torch.zeros((2 * pages - 1, 16, H, D), dtype=f8)
    whole = torch.zeros((T, Hq, D), dtype=torch.bfloat16)
    bytes_ = both.view(torch.uint8).flatten()
    for bad in (dict(q=whole, q_out=whole), dict(q_out=fused.view(-1)[:T * Hq * D].view(T, Hq, D)),
                dict(k_cache=both[:pages], v_cache=both[pages - 1:]), dict(v_cache=good["k_cache"]), dict(v_scale=good["k_scale"]),
                dict(k_cache=both[:pages], k=bytes_[:T * H * D * 2].view(torch.bfloat16).view(T, H, D)),
                dict(k_cache=both[:pages], k_scale=bytes_[:pages * H * 4].view(torch.float32).view(pages, H)),
                dict(k_cache=both[:pages], q_out=bytes_[:T * Hq * D * 2].view(torch.bfloat16).view(T, Hq, D))):
        with pytest.raises(ValueError, match="overlap"):
            bsa.bsa_append_kv_decode(**{**good, **bad})
    for ok in (dict(), dict(q_out=whole), dict(q=k, q_out=torch.zeros((T, H, D), dtype=torch.bfloat16)), dict(v=k)):
        with pytest.raises(ValueError, match="CUDA device"):
            bsa.bsa_append_kv_decode(**{**good, **ok})


def test_attention_out_apart(bsa):  # noqa: F811
    T, H, G, D, pages = 4, 2, 4, 64, 24
    f8 = torch.float8_e4m3fn
    qs = torch.zeros((T + 1, H, G, D), dtype=torch.bfloat16)
    good = dict(q=qs[:T], k_cache=torch.zeros((pages, 16, H, D), dtype=f8), v_cache=torch.zeros((pages, 16, H, D), dtype=f8),
                k_scale=torch.zeros((pages, H)), v_scale=torch.zeros((pages, H)),
                sparse_bt=torch.zeros((T, H, 8), dtype=torch.int32), sparse_ctx=torch.zeros((T, H), dtype=torch.int32))
    inside = good["v_cache"].view(torch.uint8).flatten()[:T * H * G * D * 2].view(torch.bfloat16).view(T, H, G, D)
    for bad in (dict(out=qs[1:]), dict(out=inside)):
        with pytest.raises(ValueError, match="overlap"):
            bsa.bsa_sparse_decode_attention_q8(**{**good, **bad})
    for ok in (dict(), dict(out=qs[:T]), dict(v_cache=good["k_cache"])):
        with pytest.raises(ValueError, match="CUDA device"):
            bsa.bsa_sparse_decode_attention_q8(**{**good, **ok})


def test_c_calls(bsa):  # noqa: F811
    L = bsa.lib()
    assert _rope(L, x=_at(0x1000), out=_at(0x1010)) == -2
    assert _rope(L, x=_at(0x1000), out=_at(0x1000 + 64 * 2), H=1, ts=256, ots=64) == -2
    apart = dict(k=0x100000, v=0x200000, q=0x300000, q_out=0x400000, k_cache=0x500000, v_cache=0x600000, k_scale=0x700000,
                 v_scale=0x800000)
    for bad in (dict(q_out=0x300000), dict(q_out=0x300010), dict(q_out=0x100040), dict(v_cache=0x500100), dict(k_cache=0x1FFF80),
                dict(v_scale=0x700004), dict(k_scale=0x400004)):
        a = _args(bsa, **{**apart, **bad})
        assert L.bsa_append_kv_decode(a, P16, 2, NUL) == -2
        assert L.bsa_append_kv_varlen(a, P16, P16, NUL) == -2
    far = dict(q=_at(0x100000), k=_at(0x200000), v=_at(0x300000), ks=_at(0x400000), vs=_at(0x500000))
    for out in (0x100010, 0x300040, 0x400010):
        assert _attend(L, **far, out=_at(out)) == -2
