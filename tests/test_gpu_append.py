"""Appending keys and values to the paged cache against the 64-bit oracle.

Tolerance.  Rotated keys and queries are off by the bound of the rotation
(tests/test_gpu_rope.py) before they are rounded.  A code is off by at most half a
step of its value, 2^-4 (e4m3) or 2^-3 (e5m2) of it, at least half the smallest
subnormal; a bf16 value by 2^-8.  Values (not rotated) are exact before rounding:
their codes and scales have to be equal, as have the kept codes."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
from tests.test_gpu_rope import bound

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (torch.bfloat16, 0), "e4m3": (torch.float8_e4m3fn, oracle.E4M3),
         "e5m2": (torch.float8_e5m2, oracle.E5M2)}
HALF = {0: (2.0 ** -8, 0.0), oracle.E4M3: (2.0 ** -4, 2.0 ** -10), oracle.E5M2: (2.0 ** -3, 2.0 ** -17)}


def _setup(T, H, Hq, D, B, MB, fmt, seed, amp=1.0, blocks=None):
    g = torch.Generator().manual_seed(seed)
    dtype, kind = TYPES[fmt]
    blocks = blocks or B * MB + 2
    table = torch.randperm(blocks, generator=g)[:B * MB].to(torch.int32).view(B, MB)
    qkv = (amp * torch.randn((T, Hq + 2 * H, D), generator=g)).to(torch.bfloat16)
    pages = blocks * 8
    caches = []
    for _ in range(2):
        if kind == 0:
            caches.append((torch.randn((pages, 16, H, D), generator=g).to(dtype), None))
        else:
            top = 448 if kind == oracle.E4M3 else 57344
            c = (torch.randn((pages, 16, H, D), generator=g) * top / 4).clamp(-top, top).to(dtype)
            s = torch.exp2(torch.randint(-4, 3, (pages, H), generator=g).float() + np.log2(1 / top))
            s = torch.exp2(s.log2().round())
            caches.append((c, s))
    return qkv, table, caches, dtype, kind


def _check(kind, cache, scale, want, s_want, fresh, slack, exact):
    """cache / scale from the GPU against the oracle's; `slack`: absolute
    error of a new value before rounding, in value units [num_pages, 16, H, D]
    broadcast, 0 when exact."""
    got = cache.double().cpu().numpy()
    fresh = fresh.astype(bool)
    if kind:
        sg = scale.cpu().numpy()
        assert np.array_equal(sg, s_want) if exact else np.mean(sg != s_want) < 1e-3
        same = (sg == s_want)[:, None, :, None]
        unit = s_want[:, None, :, None].astype(np.float64)
    else:
        same, unit = True, 1.0
    old = ~fresh[:, :, None, None] & same
    assert np.array_equal(np.where(old, got, 0), np.where(old, want, 0), equal_nan=True), "kept slots"
    rel, sub = HALF[kind]
    tol = np.maximum(rel * np.abs(want), sub) + slack / unit * (1 + rel)
    new = fresh[:, :, None, None] & same
    bad = new & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])
    if exact and kind:
        v = np.where(new, want, 0)
        codes = oracle.code_values(kind)[oracle.codes_of(v[fresh], kind)]
        assert np.array_equal(np.where(new, got, 0)[fresh], codes)


def _run(dev, form, qkv, H, Hq, table, caches, kind, inv, positions, axis, interleaved, rows):
    """Calls the entry point; returns (q_out, k cache, v cache, scales) on the GPU."""
    q, k, v = (t for t in qkv.to(dev).split([Hq, H, H], dim=1))
    (kc, ks), (vc, vs) = [(c.to(dev), None if s is None else s.to(dev)) for c, s in caches]
    kw = dict(q=q if Hq else None, inv_freq=None if inv is None else inv.to(dev),
              positions=None if positions is None else positions.to(dev),
              freq_axis=None if axis is None else axis.to(dev), interleaved=interleaved,
              k_scale=ks, v_scale=vs)
    if form == "decode":
        seq, dql = rows
        out = bsa.bsa_append_kv_decode(k, v, kc, vc, table.to(dev), seq.to(dev), dql, **kw)
    else:
        cu, pre = rows
        out = bsa.bsa_append_kv_varlen(k, v, kc, vc, table.to(dev), cu.to(dev), pre.to(dev), **kw)
    torch.cuda.synchronize()
    return out, kc, vc, ks, vs


def _owners(form, rows, T):
    req, pos = np.zeros(T, np.int32), np.full(T, -1, np.int64)
    if form == "decode":
        seq, dql = rows
        for t in range(T):
            req[t], pos[t] = t // dql, int(seq[t // dql]) - dql + t % dql
    else:
        cu, pre = rows
        for i in range(len(pre)):
            for t in range(int(cu[i]), int(cu[i + 1])):
                req[t], pos[t] = i, int(pre[i]) + t - int(cu[i])
    return req, pos


def _compare(dev, form, qkv, H, Hq, D, table, caches, kind, rot, axes, interleaved, rows, positions, axis):
    T = qkv.shape[0]
    inv = (1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float() if rot else None
    out, kc, vc, ks, vs = _run(dev, form, qkv, H, Hq, table, caches, kind, inv, positions, axis, interleaved, rows)
    req, pos = _owners(form, rows, T)
    place = np.maximum(pos, -1)[None].astype(np.int32) if positions is None else positions.numpy()
    q, k, v = (t.double().numpy() for t in qkv.split([Hq, H, H], dim=1))
    if rot:
        turn = lambda x: oracle.rope(x, place, inv.numpy(), None if axis is None else axis.numpy(), interleaved)  # noqa: E731
    else:
        turn = lambda x: x  # noqa: E731
    pos32 = np.clip(pos, -1, 2**31 - 1).astype(np.int32)
    if Hq:
        want_q = turn(q) * (pos >= 0)[:, None, None]
        err = np.abs(out.double().cpu().numpy() - want_q)
        assert (err <= bound(q, want_q, 1 << 20, True)).all(), err.max()
    k_fin = np.where(np.isfinite(k), k, 0)
    slack = 2 * np.abs(k_fin).max() * 3.5e-7 if rot else 0.0
    for x, cache, scale, (c0, s0), sl in ((turn(k), kc, ks, caches[0], slack), (v, vc, vs, caches[1], 0.0)):
        want, s_want, fresh = oracle.append(x, req, pos32, table.numpy(), kind, c0.double().numpy(),
                                            None if s0 is None else s0.numpy())
        _check(kind, cache, scale, want, s_want, fresh, sl, sl == 0.0)
    return out, kc, vc, ks, vs


@pytest.mark.parametrize("fmt", list(TYPES))
@pytest.mark.parametrize("B,dql,H,Hq,D,rot,inter", [
    (1, 1, 1, 1, 128, 128, False), (5, 1, 2, 6, 64, 32, True), (9, 4, 1, 8, 256, 256, False),
    (7, 3, 3, 0, 128, 0, False), (33, 2, 4, 16, 64, 64, False), (4, 40, 2, 2, 128, 30, False),
    (3, 17, 1, 5, 16, 6, True), (130, 1, 2, 4, 80, 80, False),
])
def test_append_decode(cuda_device, fmt, B, dql, H, Hq, D, rot, inter):
    """Decode rows at every slot of a page, padded requests, rows before
    position 0, scales that grow and scales that stay."""
    MB = 3
    qkv, table, caches, _, kind = _setup(B * dql, H, Hq, D, B, MB, fmt, B + D)
    g = torch.Generator().manual_seed(B)
    seq = torch.randint(0, MB * 128 + 1, (B,), generator=g, dtype=torch.int32)
    seq[::6] = 0
    seq[1::5] = 128 + 16 + dql
    _compare(cuda_device, "decode", qkv, H, Hq, D, table, caches, kind, rot, 1, inter, (seq, dql), None, None)


@pytest.mark.parametrize("fmt", list(TYPES))
@pytest.mark.parametrize("lens,pre,H,Hq,D,rot,axes", [
    ([1], [0], 1, 4, 128, 128, 1), ([16], [0], 2, 2, 64, 64, 1), ([15, 0, 17, 1], [1, 3, 31, 255], 2, 4, 128, 64, 3),
    ([300, 7, 129], [5, 120, 0], 1, 8, 128, 128, 1), ([64, 64], [64, 7], 4, 4, 256, 128, 2), ([200], [-20], 1, 1, 64, 0, 1),
])
def test_append_varlen(cuda_device, fmt, lens, pre, H, Hq, D, rot, axes):
    """Sequences of any length and start, empty ones, unowned rows before and
    behind them, explicit positions on several axes."""
    B, MB = len(lens), 4
    T = sum(lens) + 5
    qkv, table, caches, _, kind = _setup(T, H, Hq, D, B, MB, fmt, T + D)
    cu = torch.tensor([2] + lens).cumsum(0).to(torch.int32)
    g = torch.Generator().manual_seed(T)
    positions = axis = None
    if axes > 1:
        positions = torch.randint(0, 100000, (axes, T), generator=g, dtype=torch.int32)
        axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    _compare(cuda_device, "varlen", qkv, H, Hq, D, table, caches, kind, rot, axes, False,
             (cu, torch.tensor(pre, dtype=torch.int32)), positions, axis)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("amp", [0.0, 1e-39, 1e-30, 1e30])
def test_append_extreme_magnitudes(cuda_device, fmt, amp):
    """All-zero tokens (scale 1 in a fresh page), subnormal and huge values."""
    B, H, D = 6, 2, 64
    qkv, table, caches, _, kind = _setup(B * 2, H, 0, D, B, 2, fmt, 3, amp=amp)
    seq = torch.tensor([2, 18, 33, 17, 256, 100], dtype=torch.int32)
    _compare(cuda_device, "decode", qkv, H, 0, D, table, caches, kind, 0, 1, False, (seq, 2), None, None)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append_non_finite(cuda_device, fmt):
    """NaN stays NaN, infinities go to the range's end, and neither moves the
    page's scale."""
    B, H, D = 3, 1, 32
    qkv, table, caches, _, kind = _setup(B, H, 0, D, B, 1, fmt, 4)
    qkv[0, :, 5], qkv[1, :, 6], qkv[1, :, 7] = float("nan"), float("inf"), float("-inf")
    qkv[2, :, :] = float("nan")
    seq = torch.tensor([1, 4, 17], dtype=torch.int32)
    _, kc, vc, ks, vs = _run(cuda_device, "decode", qkv, H, 0, table, caches, kind, None, None, None, False, (seq, 1))
    req, pos = _owners("decode", (seq, 1), B)
    for x, cache, scale, (c0, s0) in ((qkv[:, :H], kc, ks, caches[0]), (qkv[:, H:], vc, vs, caches[1])):
        want, s_want, fresh = oracle.append(x.double().numpy(), req, pos, table.numpy(), kind, c0.double().numpy(), s0.numpy())
        assert np.array_equal(scale.cpu().numpy(), s_want)
        got = cache.double().cpu().numpy()
        at = fresh.astype(bool)
        codes = oracle.code_values(kind)[oracle.codes_of(want[at], kind)]
        assert np.array_equal(got[at], codes, equal_nan=True)


def test_append_step_by_step_fills_pages(cuda_device):
    """Forty tokens appended one by one, two by two and at once hold the same
    scales, and codes that differ at most where a subnormal was rounded twice."""
    H, D, N = 2, 64, 40
    outs = []
    for step in (1, 2, 40):
        qkv, table, caches, _, kind = _setup(N, H, 0, D, 1, 1, "e4m3", 9)
        qkv *= torch.linspace(0.1, 3.0, N).to(torch.bfloat16)[:, None, None]
        k, v = qkv.to(cuda_device).split([H, H], dim=1)
        (kc, ks), (vc, vs) = [(c.to(cuda_device), s.to(cuda_device)) for c, s in caches]
        tab = table.to(cuda_device)
        for t in range(0, N, step):
            bsa.bsa_append_kv_decode(k[t:t + step], v[t:t + step], kc, vc, tab,
                                     torch.tensor([t + step], dtype=torch.int32, device=cuda_device), step,
                                     k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        outs.append((kc.float().cpu(), ks.cpu(), vc.float().cpu(), vs.cpu()))
    for o in outs[1:]:
        assert torch.equal(o[1], outs[0][1]) and torch.equal(o[3], outs[0][3])
        for c in (0, 2):
            d = (o[c] - outs[0][c]).abs()
            assert (d <= 2.0 ** -9).all()          # one subnormal step


def test_append_bad_places_set_status(cuda_device):
    """Tokens past the table or on pages outside the cache are not stored;
    nothing else is touched; the status word says so."""
    dev = cuda_device
    B, H, D = 4, 1, 64
    qkv, table, caches, _, kind = _setup(B, H, 2, D, B, 1, "e4m3", 12, blocks=4)
    qkv = qkv[:, :2 + 2 * H]
    table = torch.tensor([[0], [-1], [4], [1]], dtype=torch.int32)
    seq = torch.tensor([5, 5, 5, 129], dtype=torch.int32)
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        _, kc, vc, ks, vs = _run(dev, "decode", qkv, H, 2, table, caches, kind, None, None, None, False, (seq, 1))
        assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID | bsa.BSA_STATUS_BAD_CONTEXT
        assert bsa.bsa_read_status() == 0
    finally:
        bsa.bsa_set_status_word(None)
    req, pos = _owners("decode", (seq, 1), B)
    for x, cache, (c0, s0) in ((qkv[:, 2:3], kc, caches[0]), (qkv[:, 3:4], vc, caches[1])):
        want, _, fresh = oracle.append(x.double().numpy(), req, pos, table.numpy(), kind, c0.double().numpy(), s0.numpy())
        assert fresh.sum() == 1
        left = ~fresh.astype(bool)
        assert np.array_equal(cache.double().cpu().numpy()[left], want[left])


def test_append_on_a_side_stream_and_in_a_graph(cuda_device):
    """A captured step replays on new inputs written into its buffers."""
    dev = cuda_device
    B, H, D = 8, 2, 128
    qkv, table, caches, _, kind = _setup(B, H, 4, D, B, 2, "e4m3", 17)
    inv = (1e4 ** (-torch.arange(32) / 32)).float().to(dev)
    buf = qkv.to(dev)
    q, k, v = buf.split([4, H, H], dim=1)
    (kc, ks), (vc, vs) = [(c.to(dev), s.to(dev)) for c, s in caches]
    seq = torch.zeros(B, dtype=torch.int32, device=dev)
    qo = torch.empty((B, 4, D), dtype=torch.bfloat16, device=dev)
    tab = table.to(dev)
    stream = torch.cuda.Stream(dev)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        bsa.bsa_append_kv_decode(k, v, kc, vc, tab, seq, 1, q=q, inv_freq=inv, k_scale=ks, v_scale=vs, q_out=qo)
    for rep in range(3):
        new = (rep + 1) * torch.randn(buf.shape, generator=torch.Generator().manual_seed(rep)).to(torch.bfloat16)
        before = [(kc.cpu(), ks.cpu()), (vc.cpu(), vs.cpu())]
        seq.copy_(torch.arange(B, dtype=torch.int32) * 31 + rep + 1)
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        rows = (seq.cpu(), 1)
        out, k2, v2, ks2, vs2 = _run(dev, "decode", new, H, 4, table, before, kind, inv.cpu(), None, None, False, rows)
        for a, b in ((qo, out), (kc, k2), (vc, v2), (ks, ks2), (vs, vs2)):
            assert torch.equal(a.float().nan_to_num(), b.float().nan_to_num())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_offsets_past_32_bits(cuda_device, fmt):
    """Pages whose elements lie past 2^32 in the cache; an empty call."""
    dev = cuda_device
    H, D, B = 4, 256, 5
    qkv, table, caches, dtype, kind = _setup(B, H, 3, D, B, 1, fmt, 23)
    seq = torch.tensor([1, 17, 128, 40, 9], dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(64) / 64)).float()
    out, kc, vc, ks, vs = _run(dev, "decode", qkv, H, 3, table, caches, kind, inv, None, None, False, (seq, 1))
    small = kc.shape[0]
    pages = (1 << 32) // (16 * H * D) // 8 * 8 + small
    base = (pages - small) // 8
    far = torch.empty((2, pages, 16, H, D), dtype=dtype, device=dev)
    fars = torch.empty((2, pages, H), device=dev) if kind else None
    for i, (c, s) in enumerate(caches):
        far[i].view(torch.uint8)[pages - small:] = c.to(dev).view(torch.uint8)
        if kind:
            fars[i, pages - small:] = s.to(dev)
    q, k, v = qkv.to(dev).split([3, H, H], dim=1)
    args = dict(q=q, inv_freq=inv.to(dev), k_scale=fars[0] if kind else None, v_scale=fars[1] if kind else None)
    got = bsa.bsa_append_kv_decode(k, v, far[0], far[1], (table + base).to(dev), seq.to(dev), 1, **args)
    torch.cuda.synchronize()
    assert torch.equal(got, out)
    for a, b in ((far[0], kc), (far[1], vc)):
        assert torch.equal(a.view(torch.uint8)[pages - small:], b.view(torch.uint8))
    if kind:
        assert torch.equal(fars[0, pages - small:], ks) and torch.equal(fars[1, pages - small:], vs)
    none = bsa.bsa_append_kv_decode(k[:0], v[:0], far[0], far[1], table[:0].to(dev), seq[:0].to(dev), 1,
                                    **{**args, "q": q[:0]})
    assert none.shape == (0, 3, D)


def test_append_strides_of_single_entries_do_not_matter(cuda_device):
    """One token, one head: whatever strides its dimensions of one entry have."""
    dev = cuda_device
    D = 64
    qkv, table, caches, _, kind = _setup(1, 1, 1, D, 1, 1, "e4m3", 31)
    seq = torch.tensor([7], dtype=torch.int32)
    out, kc, vc, ks, vs = _run(dev, "decode", qkv, 1, 1, table, caches, kind, None, None, None, False, (seq, 1))
    odd = [t.to(dev).contiguous().as_strided((1, 1, D), (5, 3, 1)) for t in qkv.split([1, 1, 1], dim=1)]
    (k2, s2), (v2, t2) = [(c.to(dev), s.to(dev)) for c, s in caches]
    got = bsa.bsa_append_kv_decode(odd[1], odd[2], k2, v2, table.to(dev), seq.to(dev), 1, q=odd[0], k_scale=s2, v_scale=t2)
    torch.cuda.synchronize()
    for a, b in ((got, out), (k2, kc), (v2, vc), (s2, ks), (t2, vs)):
        assert torch.equal(a.float().nan_to_num(), b.float().nan_to_num())


@pytest.mark.parametrize("fmt", list(TYPES))
@pytest.mark.parametrize("lens,pre,H,Hq,D,rot,axes", [
    ([15, 0, 17, 1], [1, 3, 31, 255], 2, 4, 128, 104, 3), ([300, 7, 129], [5, 120, 0], 1, 3, 80, 72, 1),
    ([1], [47], 1, 8, 64, 24, 1), ([64, 33], [64, 7], 3, 0, 256, 232, 2), ([200], [-20], 1, 1, 16, 8, 1),
    ([311] * 17, list(range(17)), 1, 2, 64, 56, 1),
])
def test_append_pairs_at_multiples_of_four(cuda_device, fmt, lens, pre, H, Hq, D, rot, axes):
    """Half-split pairs whose distance is a multiple of 4 and not of 8, in short
    calls and in one with 16 rows per CTA."""
    assert rot // 2 % 8 == 4
    B, MB = len(lens), 4
    T = sum(lens) + 5
    qkv, table, caches, _, kind = _setup(T, H, Hq, D, B, MB, fmt, T + D + rot)
    cu = torch.tensor([2] + lens).cumsum(0).to(torch.int32)
    g = torch.Generator().manual_seed(T)
    positions = axis = None
    if axes > 1:
        positions = torch.randint(0, 100000, (axes, T), generator=g, dtype=torch.int32)
        axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    _compare(cuda_device, "varlen", qkv, H, Hq, D, table, caches, kind, rot, axes, False,
             (cu, torch.tensor(pre, dtype=torch.int32)), positions, axis)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [323, 324, 647, 1293, 2584, 2590, 3000, 5168, 5175, 9000])
def test_append_calls_of_every_length(cuda_device, fmt, T):
    """One KV head in calls on both sides of each number of rows per CTA."""
    lens = [449] * (T // 449) + [T % 449]
    pre = [(7 * i) % 60 for i in range(len(lens))]
    qkv, table, caches, _, kind = _setup(T + 5, 1, 1, 16, len(lens), 4, fmt, T)
    cu = torch.tensor([2] + lens).cumsum(0).to(torch.int32)
    _compare(cuda_device, "varlen", qkv, 1, 1, 16, table, caches, kind, 16, 1, False,
             (cu, torch.tensor(pre, dtype=torch.int32)), None, None)
