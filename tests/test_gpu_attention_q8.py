"""Sparse decode attention over the 8-bit cache against the 64-bit oracle.

Tolerance.  With A = sum_j p_j |v_j| (the oracle on the values' magnitudes):
probabilities may be held as two 8-bit terms of 4 significant bits each, off
by at most 2^-8 of each; a score is off by at most D 2^-24 sum |q k| scale
(below 2^-10 for the sizes here), which moves each probability and their sum
by as much; bf16 rounds the output by half a step, 2^-8 of it.
|error| <= 2^-8 |out| + (2^-8 + 2 * 2^-10) (1 + 2^-8) A."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
import synth

pytestmark = pytest.mark.gpu

KIND = {"e4m3": (torch.float8_e4m3fn, oracle.E4M3, 448.0), "e5m2": (torch.float8_e5m2, oracle.E5M2, 57344.0)}


def _case(T, H, G, D, K, fmt, ctx, seed, pages=None, amp=1.0):
    """Random pages for each row; slots that no row attends to hold NaN codes."""
    dtype, kind, top = KIND[fmt]
    g = torch.Generator().manual_seed(seed)
    W = K * 8
    pages = pages or T * H * W + 3
    used = T * H * W
    perm = torch.randperm(max(pages, used), generator=g) % pages
    bt = perm[:used].view(T, H, W).to(torch.int32)
    ctx = torch.as_tensor(ctx, dtype=torch.int32).view(T, H)
    c, s = [], []
    for _ in range(2):
        x = torch.randn((pages, 16, H, D), generator=g)
        s.append(torch.exp2(torch.randint(-2, 2, (pages, H), generator=g).float()) * 4.5 / top)
        c.append((x * top / 4.5).clamp(-top, top).to(dtype).view(torch.uint8))
    if pages >= used:
        live = torch.zeros((pages, 16, H), dtype=torch.bool)
        j = torch.arange(W * 16)
        for t in range(T):
            for h in range(H):
                n = int(ctx[t, h].clamp(0, W * 16))
                live[bt[t, h, j[:n] // 16].long(), j[:n] % 16, h] = True
        for x in c:
            x[~live] = 0x7F
    q = (amp * torch.randn((T, H, G, D), generator=g)).to(torch.bfloat16)
    return q, c, s, bt, ctx, dtype, kind


def _bound(q, c, s, bt, ctx, kind, scale, want):
    mag = oracle.sparse_decode_attention_q8(q, c[0], c[1] & 0x7F, kind, s[0], s[1], bt, ctx, scale)
    return 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 1e-30


def _check(dev, q, c, s, bt, ctx, dtype, kind, scale=None):
    sc = q.shape[-1] ** -0.5 if scale is None else scale
    cn, sn = [x.numpy() for x in c], [x.numpy() for x in s]
    want = oracle.sparse_decode_attention_q8(q, cn[0], cn[1], kind, sn[0], sn[1], bt.numpy(), ctx.numpy(), sc)
    got = bsa.bsa_sparse_decode_attention_q8(
        q.to(dev), c[0].to(dev).view(dtype), c[1].to(dev).view(dtype), s[0].to(dev), s[1].to(dev),
        bt.to(dev), ctx.to(dev), scale=scale)
    torch.cuda.synchronize()
    g = got.double().cpu().numpy()
    tol = _bound(q, cn, sn, bt.numpy(), ctx.numpy(), kind, sc, want)
    assert np.isfinite(g).all()
    bad = np.abs(g - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:3], want[bad][:3], tol[bad][:3], bad.mean())
    return got


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("T,H,G,D,K,ctx", [
    (1, 1, 1, 128, 1, [1]), (1, 1, 8, 128, 1, [128]), (2, 2, 4, 64, 2, [0, 15, 16, 17]),
    (3, 1, 16, 128, 4, [127, 129, 512]), (2, 1, 5, 256, 3, [300, 33]), (1, 3, 3, 64, 16, [2048, 1999, 2]),
    (4, 2, 8, 128, 16, [2048, 1, 1025, 1024, 0, 1023, 1900, 64]), (2, 1, 9, 64, 5, [640, 639]),
    (2, 1, 2, 256, 17, [2176, 2049]), (1, 2, 16, 256, 9, [1152, 1000]), (5, 1, 7, 128, 20, [2560, 100, 2057, 0, 1281]),
    (1, 1, 4, 128, 64, [8192]), (2, 1, 8, 64, 40, [5000, 5120]),
])
def test_attention_q8(cuda_device, fmt, T, H, G, D, K, ctx):
    _check(cuda_device, *_case(T, H, G, D, K, fmt, ctx, T + G + D + K))


@pytest.mark.parametrize("amp", [0.0, 1e-3, 30.0])
def test_attention_q8_flat_and_peaked(cuda_device, amp):
    """All-equal scores; almost one-hot rows (large scores: the score bound is
    scaled with them)."""
    q, c, s, bt, ctx, dtype, kind = _case(3, 1, 4, 128, 8, "e4m3", [1024, 777, 3], 40, amp=amp)
    if amp < 1:
        _check(cuda_device, q, c, s, bt, ctx, dtype, kind)
        return
    got = bsa.bsa_sparse_decode_attention_q8(
        *(x.to(cuda_device) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)))
    want = oracle.sparse_decode_attention_q8(q, c[0].numpy(), c[1].numpy(), kind, s[0].numpy(), s[1].numpy(),
                                             bt.numpy(), ctx.numpy(), 128 ** -0.5)
    tol = _bound(q, [x.numpy() for x in c], [x.numpy() for x in s], bt.numpy(), ctx.numpy(), kind, 128 ** -0.5, want)
    mag = float(c[1].view(dtype).float().nan_to_num().abs().max() * s[1].max())
    # |score| <= amp * 20 here: D 2^-24 sum |q k| scale <= 2^-17 * 30 * 100
    assert (np.abs(got.double().cpu().numpy() - want) <= tol + 2 * 2.0 ** -17 * 3000 * mag).all()


def test_attention_q8_scales_far_apart(cuda_device):
    """Pages whose value scales differ by 2^40, scales that are no powers of two."""
    q, c, s, bt, ctx, dtype, kind = _case(2, 2, 4, 64, 4, "e4m3", [512, 500, 17, 333], 50)
    s[1] *= torch.exp2(torch.randint(-20, 21, s[1].shape, generator=torch.Generator().manual_seed(1)).float())
    s[0] *= 0.7
    s[1] *= 1.3
    _check(cuda_device, q, c, s, bt, ctx, dtype, kind)


def test_attention_q8_queries_with_wide_range(cuda_device):
    """Query values from 2^-20 to 1 in one head, and heads far apart."""
    q, c, s, bt, ctx, dtype, kind = _case(2, 1, 8, 128, 4, "e4m3", [512, 300], 51)
    g = torch.Generator().manual_seed(3)
    q = (q.float() * torch.exp2(-20 * torch.rand(q.shape, generator=g))).to(torch.bfloat16)
    q[:, :, 1] *= 2.0 ** -60
    q[:, :, 2] = 0
    q[:, :, 3] *= 8
    _check(cuda_device, q, c, s, bt, ctx, dtype, kind)


def test_attention_q8_pages_out_of_range_and_status(cuda_device):
    """Tokens on pages outside the cache take no part; a row of only such pages
    gives zeros; contexts are clamped; the status word says so."""
    dev = cuda_device
    q, c, s, bt, ctx, dtype, kind = _case(4, 1, 3, 128, 3, "e4m3", [384, 100, 50, 384], 60, pages=50)
    bt[0, 0, 3], bt[0, 0, 7], bt[0, 0, 11] = -1, 50, 2**31 - 1
    bt[1, 0, :7] = torch.tensor([60, -5, 50, 51, 1000, -2**31, 99])
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        got = _check(dev, q, c, s, bt, ctx, dtype, kind)
        assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_PAGE
        assert (got[1] == 0).all()
        bt.clamp_(0, 49)
        ctx[2, 0], ctx[3, 0] = -7, 385
        got = _check(dev, q, c, s, bt, ctx, dtype, kind)
        assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_CONTEXT
        assert (got[2] == 0).all()
        ctx.clamp_(0, 384)
        _check(dev, q, c, s, bt, ctx, dtype, kind)
        assert bsa.bsa_read_status() == 0
    finally:
        bsa.bsa_set_status_word(None)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_q8_nan_in_and_outside_the_context(cuda_device, D):
    """A NaN value in the context reaches its dimension of the row's heads and
    nothing else; NaN in the slots behind the context reaches nothing (the
    cases above hold it there); a NaN key poisons its row."""
    q, c, s, bt, ctx, dtype, kind = _case(3, 1, 2, D, 2, "e4m3", [200, 131, 9], 70)
    c[1][bt[0, 0, 5], 3, 0, 17] = 0xFF
    c[0][bt[2, 0, 0], 4, 0, 1] = 0x7F
    got = bsa.bsa_sparse_decode_attention_q8(
        *(x.to(cuda_device) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)))
    bad = torch.isnan(got.cpu())
    want = torch.zeros_like(bad)
    want[0, 0, :, 17] = True
    want[2] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T,H,G,D,K,n", [(3, 2, 8, 128, 128, 16000), (1, 1, 16, 64, 1024, 131072), (1, 1, 2, 256, 300, 38399),
                                         (40, 2, 4, 64, 48, 6000)])
def test_attention_q8_long_rows(cuda_device, T, H, G, D, K, n):
    """Few long rows: the work over one row is split and joined."""
    ctx = [max(0, n - 1237 * i) for i in range(T * H)]
    _check(cuda_device, *_case(T, H, G, D, K, "e4m3", ctx, 80 + D, pages=2000))


def test_attention_q8_shared_blocks_many_rows(cuda_device):
    """More rows than CTAs fit, all on the same few pages."""
    T = 700
    g = torch.Generator().manual_seed(2)
    ctx = torch.randint(0, 385, (T, 1), generator=g)
    _check(cuda_device, *_case(T, 1, 4, 64, 3, "e5m2", ctx, 90, pages=40))


def test_attention_q8_streams_workspace_and_graph(cuda_device):
    """The same bits on a side stream, with a caller's workspace full of old
    bytes, and from a captured graph replayed on other inputs."""
    dev = cuda_device
    q, c, s, bt, ctx, dtype, kind = _case(2, 2, 8, 128, 64, "e4m3", [8192, 8000, 100, 4097], 95, pages=900)
    args = [x.to(dev) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)]
    ref = bsa.bsa_sparse_decode_attention_q8(*args)
    torch.cuda.synchronize()
    need = bsa.bsa_attention_q8_workspace_bytes(2, 2, 8, 128, 64)
    stream = torch.cuda.Stream(dev)
    with torch.cuda.stream(stream):
        a = bsa.bsa_sparse_decode_attention_q8(*args)
        ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device=dev)
        b = bsa.bsa_sparse_decode_attention_q8(*args, workspace=ws[:need])
        b2 = bsa.bsa_sparse_decode_attention_q8(*args, workspace=ws[:need])
    stream.synchronize()
    assert torch.equal(a, ref) and torch.equal(b, ref) and torch.equal(b2, ref)
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        bsa.bsa_sparse_decode_attention_q8(*args, out=out)
    for rep in range(3):
        q2 = synth.normal_scores(q.shape, torch.bfloat16, seed=rep)
        args[0].copy_(q2)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, bsa.bsa_sparse_decode_attention_q8(*args))
    assert torch.equal(args[0].cpu(), q2)


def test_attention_q8_refuses_small_or_misaligned_workspaces(cuda_device):
    dev = cuda_device
    q, c, s, bt, ctx, dtype, kind = _case(1, 1, 8, 128, 256, "e4m3", [32768], 97, pages=300)
    args = [x.to(dev) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)]
    need = bsa.bsa_attention_q8_workspace_bytes(1, 1, 8, 128, 256)
    if need == 0:
        return
    ws = torch.empty(need + 512, dtype=torch.uint8, device=dev)
    for bad in (ws[:need - 1], ws[16:]):
        with pytest.raises(bsa.BsaError) as e:
            bsa.bsa_sparse_decode_attention_q8(*args, workspace=bad)
        assert e.value.status == -5


@pytest.mark.parametrize("H,G,D,fmt", [(1, 4, 64, "e4m3"), (2, 8, 128, "e5m2"), (1, 3, 256, "e4m3"), (2, 16, 128, "e4m3")])
def test_attention_q8_blocks_in_runs(cuda_device, H, G, D, fmt):
    """Tables as the selector writes them: a block's eight pages follow one
    another (the last block of the cache among them), mixed with blocks whose
    pages almost do."""
    T, K, blocks = 5, 9, 60
    q, c, s, bt, _, dtype, kind = _case(T, H, G, D, K, fmt, [0] * (T * H), 30 + D, pages=blocks * 8)
    for x in c:                          # no NaN codes: every page is read somewhere
        x[(x & 0x7F) == 0x7F] = 0x3A
    g = torch.Generator().manual_seed(D)
    phys = torch.stack([torch.randperm(blocks, generator=g)[:K] for _ in range(T * H)]).view(T, H, K)
    phys[0, 0, 3] = blocks - 1
    bt = (phys[..., None] * 8 + torch.arange(8)).view(T, H, K * 8).to(torch.int32)
    bt[1, 0, 16:24] = bt[1, 0, 16:24].flip(0)
    bt[1, 0, 31] += 1 if bt[1, 0, 31] < blocks * 8 - 1 else -1
    bt[2, 0, 8:16] = torch.arange(blocks * 8 - 4, blocks * 8 + 4)      # runs out of the cache
    ctx = torch.tensor([K * 128, 1100, 1027, 897, 128, 15, 1, 1151, 1040, 640][:T * H], dtype=torch.int32).view(T, H)
    _check(cuda_device, q, c, s, bt, ctx, dtype, kind)


def test_attention_q8_empty_cache_and_empty_batch(cuda_device):
    """No page at all: every token's page is out of range, so zeros; no rows:
    nothing is launched."""
    dev = cuda_device
    q = synth.normal_scores((3, 2, 4, 128), torch.bfloat16, seed=1).to(dev)
    kc = torch.empty((0, 16, 2, 128), dtype=torch.float8_e4m3fn, device=dev)
    sc = torch.empty((0, 2), device=dev)
    bt = torch.zeros((3, 2, 16), dtype=torch.int32, device=dev)
    ctx = torch.full((3, 2), 200, dtype=torch.int32, device=dev)
    got = bsa.bsa_sparse_decode_attention_q8(q, kc, kc, sc, sc, bt, ctx)
    torch.cuda.synchronize()
    assert (got == 0).all()
    none = bsa.bsa_sparse_decode_attention_q8(q[:0], kc, kc, sc, sc, bt[:0], ctx[:0])
    assert none.shape == (0, 2, 4, 128)


def test_attention_q8_offsets_past_32_bits(cuda_device):
    """Pages whose bytes lie past 2^32 in the cache."""
    dev = cuda_device
    H, D, G, K = 4, 256, 4, 2
    pages = (1 << 32) // (16 * H * D) + 100
    q, c, s, bt, ctx, dtype, kind = _case(2, H, G, D, K, "e4m3", [256, 200, 17, 128, 1, 255, 100, 31], 5)
    small = c[0].shape[0]
    far = torch.empty((2, pages, 16, H, D), dtype=torch.uint8, device=dev)
    fars = torch.empty((2, pages, H), device=dev)
    for i in range(2):
        far[i, pages - small:] = c[i].to(dev)
        fars[i, pages - small:] = s[i].to(dev)
    near = _check(dev, q, c, s, bt, ctx, dtype, kind)
    got = bsa.bsa_sparse_decode_attention_q8(q.to(dev), far[0].view(dtype), far[1].view(dtype), fars[0], fars[1],
                                             (bt + pages - small).to(dev), ctx.to(dev))
    torch.cuda.synchronize()
    assert torch.equal(got, near)


@pytest.mark.parametrize("T,H,G,D,K,joins", [(1, 1, 8, 128, 16, "cluster"), (3, 1, 12, 64, 8, "cluster"), (2, 1, 3, 256, 2, "cluster"),
                                             (1, 2, 8, 64, 512, "launch"), (1, 1, 16, 128, 1024, "launch")])
def test_attention_q8_joined_rows_in_a_graph(cuda_device, T, H, G, D, K, joins):
    """Rows joined by their cluster, or by a launch with a workspace, captured and
    replayed on contexts of all lengths, empty shares among them."""
    dev = cuda_device
    q, c, s, bt, ctx, dtype, kind = _case(T, H, G, D, K, "e4m3", [K * 128] * (T * H), 7, pages=700)
    for x in c:                          # no NaN codes: every page is read somewhere
        x[(x & 0x7F) == 0x7F] = 0x31
    assert (bsa.bsa_attention_q8_workspace_bytes(T, H, G, D, K) > 0) == (joins == "launch")
    args = [x.to(dev) for x in (q, c[0].view(dtype), c[1].view(dtype), s[0], s[1], bt, ctx)]
    out = torch.empty_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream(dev)):
        bsa.bsa_sparse_decode_attention_q8(*args, out=out)
    for n in (K * 128, 1, 0, 129, K * 64 + 5, 3 * 128):
        n = min(n, K * 128)
        args[6].fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = _check(dev, q, c, s, bt, torch.full_like(ctx, n), dtype, kind)
        assert torch.equal(got, want), n
