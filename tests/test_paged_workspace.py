"""A caller's workspace that lies over another argument is refused (no GPU: nothing here
launches a kernel, as every call is one that is refused)."""
import ctypes

import pytest

from tests.test_paged_abi import NUL, _args, _blocks, bsa  # noqa: F401

HUGE = 1 << 40


SIZES = {"q": 8 * 2 * 4 * 64 * 2, "out": 8 * 2 * 4 * 64 * 2, "k_cache": 64 * 16 * 2 * 64, "v_cache": 64 * 16 * 2 * 64,
         "k_scale": 64 * 2 * 4, "v_scale": 64 * 2 * 4, "block_table": 4 * 2 * 4, "rows": 4 * 4, "cu": 5 * 4}


@pytest.mark.parametrize("form,what", [(f, w) for f in ("decode", "varlen") for w in SIZES if (f, w) != ("decode", "cu")])
def test_paged_attention(bsa, form, what):      # noqa: F811
    """The workspace begins in the argument's last bytes, or ends in its first."""
    L = bsa.lib()
    need = bsa.bsa_paged_attention_workspace_bytes(8, 2, 4, 64)
    assert need > 0
    # every argument far from the others, in places of 2^40 bytes
    place = dict(q=1, out=2, k_cache=3, v_cache=4, k_scale=5, v_scale=6, block_table=7, rows=8, cu=9)
    at = {k: n * HUGE + 8 * 256 - 256 for k, n in place.items()}
    for ws in (at[what] // 256 * 256 + (SIZES[what] - 1) // 256 * 256, at[what] // 256 * 256 - need + 256):
        assert ws % 256 == 0
        a = _args(bsa, **{k: v for k, v in at.items() if k not in ("rows", "cu")}, workspace=ws, workspace_bytes=need)
        rows, cu = (ctypes.c_void_p(at[k]) for k in ("rows", "cu"))
        got = L.bsa_paged_attention_decode(a, rows, 2, NUL) if form == "decode" else L.bsa_paged_attention_varlen(a, cu, rows, NUL)
        assert got == -2
        # a workspace that is too small is that first
        a.workspace_bytes = need - 1
        got = L.bsa_paged_attention_decode(a, rows, 2, NUL) if form == "decode" else L.bsa_paged_attention_varlen(a, cu, rows, NUL)
        assert got == -5


NAMES = ["table", "lens", "refs", "parent", "more", "out0", "out1", "out2", "tensor0", "tensor1"]


@pytest.mark.parametrize("call,what", [(c, w) for c in ("fork", "compact") for w in NAMES if c == "fork" or w not in ("parent", "more")])
def test_blocks(bsa, call, what):      # noqa: F811
    L = bsa.lib()
    need = L.bsa_fork_workspace_bytes(4, 4, 2, 64) if call == "fork" else L.bsa_compact_workspace_bytes(64)
    at = {k: (i + 1) * HUGE for i, k in enumerate(NAMES)}
    for ws in (at[what], at[what] - 256):
        got = _blocks(bsa, call, tensors=((at["tensor0"], 64), (at["tensor1"], 4096)), table=at["table"], lens=at["lens"], refs=at["refs"],
                      parent=at["parent"], more=at["more"], o=(at["out0"], at["out1"], at["out2"]), ws=ws, wb=need)
        assert got == -2, ws
    got = _blocks(bsa, call, tensors=((at["tensor0"], 64),), ws=at[what], wb=255)
    assert got == -5
