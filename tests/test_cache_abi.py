"""Host-side argument checks of the rotary, append and 8-bit attention calls
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
P16 = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


def _rope(L, x=P16, dtype=0, T=4, H=2, D=64, ts=128, hs=64, pos=P16, axes=1, inv=P16, axis=NUL,
          rot=64, flags=0, out=P16, ots=128, ohs=64):
    return L.bsa_rope(x, dtype, T, H, D, ts, hs, pos, axes, inv, axis, rot, flags, out, ots, ohs, NUL)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=2), -4), (dict(T=-1), -2), (dict(D=0), -2), (dict(D=2000, rot=64), -2),
    (dict(rot=63), -2), (dict(rot=66), -2), (dict(rot=-2), -2), (dict(axes=0), -2),
    (dict(axes=9, axis=P16), -2), (dict(flags=4), -2), (dict(axes=3), -1), (dict(pos=NUL), -1),
    (dict(inv=NUL), -1), (dict(x=NUL), -1), (dict(out=NUL), -1), (dict(ots=100), -2),
    (dict(ohs=60), -2), (dict(ots=-128), -2), (dict(ts=-1), -2), (dict(x=ctypes.c_void_p(0x1001)), -7),
    (dict(dtype=1, out=ODD), -7), (dict(ts=256), -2), (dict(T=0, x=NUL, out=NUL, pos=NUL), 0),
])
def test_rope_refusals(bsa, bad, code):
    assert _rope(bsa.lib(), **bad) == code


def _args(bsa, **kw):
    a = bsa.AppendArgs()
    d = dict(k=0x1000, v=0x1000, q=0x1000, T=8, H=2, Hq=4, D=64, k_token_stride=128,
             k_head_stride=64, v_token_stride=128, v_head_stride=64, q_token_stride=256,
             q_head_stride=64, q_out=0x1000, positions=0, inv_freq=0x1000, freq_axis=0, axes=1,
             rot_dim=64, flags=0, cache_dtype=2, k_cache=0x1000, v_cache=0x1000, num_pages=64,
             k_scale=0x1000, v_scale=0x1000, block_table=0x1000, num_reqs=4, max_blocks=2)
    d.update(kw)
    for k, v in d.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad,code", [
    (dict(cache_dtype=1), -4), (dict(T=-1), -2), (dict(H=0), -2), (dict(D=72), -2),
    (dict(D=272), -2), (dict(num_pages=-1), -2), (dict(max_blocks=1 << 24), -2),
    (dict(k_token_stride=-8), -2), (dict(k_token_stride=132), -7), (dict(q_head_stride=60), -7),
    (dict(q_out=0), -1), (dict(q=0), -1), (dict(rot_dim=66), -2), (dict(rot_dim=3), -2),
    (dict(inv_freq=0), -1), (dict(axes=2), -1), (dict(axes=2, freq_axis=0x1000), -1),
    (dict(k=0), -1), (dict(v_cache=0), -1), (dict(k_scale=0), -1), (dict(block_table=0), -1),
    (dict(k=0x1008), -7), (dict(k_cache=0x1004), -7), (dict(v_scale=0x1002), -7), (dict(q_out=0x1008), -7),
])
def test_append_refusals(bsa, bad, code):
    L = bsa.lib()
    a = _args(bsa, **bad)
    assert L.bsa_append_kv_decode(a, P16, 2, NUL) == code
    assert L.bsa_append_kv_varlen(a, P16, P16, NUL) == code


def test_append_form_refusals(bsa):
    L = bsa.lib()
    assert L.bsa_append_kv_decode(None, P16, 2, NUL) == -1
    assert L.bsa_append_kv_decode(_args(bsa), P16, 3, NUL) == -6
    assert L.bsa_append_kv_decode(_args(bsa), P16, 0, NUL) == -2
    assert L.bsa_append_kv_decode(_args(bsa), NUL, 2, NUL) == -1
    assert L.bsa_append_kv_varlen(_args(bsa), NUL, P16, NUL) == -1
    assert L.bsa_append_kv_varlen(_args(bsa), P16, NUL, NUL) == -1
    empty = _args(bsa, T=0, num_reqs=0, k=0, v=0, q=0, q_out=0, k_cache=0, v_cache=0, num_pages=0)
    assert L.bsa_append_kv_decode(empty, NUL, 1, NUL) == 0
    assert L.bsa_append_kv_varlen(empty, NUL, NUL, NUL) == 0


def _attend(L, q=P16, k=P16, v=P16, dtype=2, ks=P16, vs=P16, pages=64, bt=P16, ctx=P16, T=2, H=2,
            G=4, D=64, K=16, out=P16, ws=NUL, wb=0):
    return L.bsa_sparse_decode_attention_q8(q, k, v, dtype, ks, vs, pages, bt, ctx, T, H, G, D, K,
                                            0.1, out, ws, wb, NUL)


@pytest.mark.parametrize("bad,code", [
    (dict(dtype=0), -4), (dict(dtype=1), -4), (dict(T=-1), -2), (dict(H=0), -2), (dict(G=0), -2),
    (dict(G=17), -2), (dict(D=96), -2), (dict(D=512), -2), (dict(K=0), -3), (dict(K=1025), -3),
    (dict(pages=-1), -2), (dict(pages=1 << 27), -2), (dict(q=NUL), -1), (dict(k=NUL), -1),
    (dict(vs=NUL), -1), (dict(bt=NUL), -1), (dict(out=NUL), -1), (dict(q=ODD), -7),
    (dict(v=ODD), -7), (dict(out=ODD), -7), (dict(T=0, q=NUL), 0),
])
def test_attention_q8_refusals(bsa, bad, code):
    assert _attend(bsa.lib(), **bad) == code


def test_binding_refuses_before_any_launch(bsa):
    """Wrong shapes, types, devices and strides raise ValueError naming the
    argument; the arguments that pass end at the check that they are on a GPU
    (CPU tensors stand in for device tensors, so nothing can be launched)."""

    def t(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)

    def refuses(fn, good, bad, match):
        with pytest.raises(ValueError, match="CUDA device"):
            fn(**good)
        for name, value in bad:
            with pytest.raises((ValueError, TypeError), match=match.get(name, name)):
                fn(**{**good, name: value})

    i32, f32, f8 = torch.int32, torch.float32, torch.float8_e4m3fn
    meta = torch.empty((5,), dtype=i32, device="meta")
    refuses(bsa.bsa_rope, dict(x=t(5, 3, 64), positions=t(5, dtype=i32), inv_freq=t(32, dtype=f32)), [
        ("x", t(5, 64)), ("x", t(5, 3, 64, dtype=torch.float16)), ("x", t(5, 64, 3).transpose(1, 2)),
        ("x", None), ("x", 3), ("positions", t(4, dtype=i32)), ("positions", t(5, dtype=torch.int64)),
        ("positions", t(3, 4, dtype=i32)), ("positions", t(1, 1, 5, dtype=i32)), ("positions", None),
        ("positions", t(10, dtype=i32)[::2]), ("positions", meta), ("inv_freq", None),
        ("inv_freq", t(32, dtype=torch.float64)), ("inv_freq", t(32, 1, dtype=f32)),
        ("freq_axis", t(31, dtype=i32)), ("out", t(5, 2, 64)), ("out", t(5, 3, 64, dtype=f32)),
    ], {})
    with pytest.raises(ValueError, match="freq_axis"):
        bsa.bsa_rope(t(5, 3, 64), t(2, 5, dtype=i32), t(32, dtype=f32))
    good = dict(k=t(6, 2, 64), v=t(6, 2, 64), k_cache=t(24, 16, 2, 64, dtype=f8),
                v_cache=t(24, 16, 2, 64, dtype=f8), block_table=t(3, 4, dtype=i32), q=t(6, 8, 64),
                q_out=t(6, 8, 64), inv_freq=t(32, dtype=f32), k_scale=t(24, 2, dtype=f32),
                v_scale=t(24, 2, dtype=f32))
    bad = [("k", t(6, 2, 64, dtype=f32)), ("v", t(6, 3, 64)), ("v", t(5, 2, 64)), ("q", t(6, 8, 32)),
           ("q_out", t(6, 7, 64)), ("q", None), ("k_cache", t(24, 8, 2, 64, dtype=f8)),
           ("k_cache", t(24, 16, 2, 64, dtype=f32)), ("v_cache", t(23, 16, 2, 64, dtype=f8)),
           ("v_cache", t(24, 16, 2, 64)), ("k_scale", None), ("v_scale", t(24, 1, dtype=f32)),
           ("block_table", t(2, 4, dtype=i32)), ("block_table", t(3, 4)), ("positions", t(2, 5, dtype=i32)),
           ("positions", meta)]
    match = {"k_cache": "cache", "q": "q"}
    refuses(bsa.bsa_append_kv_decode, dict(good, seq_lens=t(3, dtype=i32), decode_query_len=2),
            bad + [("seq_lens", t(3, 1, dtype=i32)), ("seq_lens", None), ("decode_query_len", 2.0)],
            dict(match, decode_query_len="float"))
    refuses(bsa.bsa_append_kv_varlen, dict(good, cu_seqlens_q=t(4, dtype=i32), prefix_lens=t(3, dtype=i32)),
            bad + [("cu_seqlens_q", t(3, dtype=i32)), ("cu_seqlens_q", 4), ("prefix_lens", t(3))], match)
    with pytest.raises(ValueError, match="bfloat16 cache"):
        bsa.bsa_append_kv_decode(**dict(good, k_cache=t(24, 16, 2, 64), v_cache=t(24, 16, 2, 64)),
                                 seq_lens=t(3, dtype=i32), decode_query_len=2)
    refuses(bsa.bsa_sparse_decode_attention_q8,
            dict(q=t(6, 2, 4, 64), k_cache=good["k_cache"], v_cache=good["v_cache"], k_scale=good["k_scale"],
                 v_scale=good["v_scale"], sparse_bt=t(6, 2, 32, dtype=i32), sparse_ctx=t(6, 2, dtype=i32)),
            [("q", t(6, 2, 64)), ("q", t(6, 2, 4, 64, dtype=f32)), ("q", t(6, 2, 64, 4).transpose(2, 3)),
             ("k_cache", t(24, 16, 2, 64)), ("v_cache", t(24, 16, 2, 32, dtype=f8)),
             ("v_cache", t(24, 16, 2, 64, dtype=torch.float8_e5m2)), ("k_scale", None),
             ("v_scale", t(23, 2, dtype=f32)), ("sparse_bt", t(6, 2, 30, dtype=i32)),
             ("sparse_bt", t(6, 1, 32, dtype=i32)), ("sparse_ctx", t(6, dtype=i32)), ("out", t(6, 2, 4, 32)),
             ("out", t(6, 2, 4, 64, dtype=f32)), ("scale", "x")], dict(match, scale="number"))
    bf = t(24, 16, 2, 64)
    with pytest.raises(ValueError, match="float8"):
        bsa.bsa_sparse_decode_attention_q8(t(6, 2, 4, 64), bf, bf, None, None, t(6, 2, 32, dtype=i32),
                                           t(6, 2, dtype=i32))
