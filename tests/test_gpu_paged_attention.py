"""Attention of new tokens over the whole paged cache against the 64-bit oracle.

Tolerance.  With A = sum_j p_j |v_j| (the oracle on the values' magnitudes):
probabilities (times a page's scale) are rounded to bf16 once, off by at most
2^-8 of each; a score is off by at most D 2^-24 sum |q k| scale (below 2^-10
for the sizes here), which moves each probability and their sum by as much;
bf16 rounds the output by half a step, 2^-8 of it.
|error| <= 2^-8 |out| + (2^-8 + 2 * 2^-10) (1 + 2^-8) A."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle

pytestmark = pytest.mark.gpu

KIND = {"bf16": (torch.bfloat16, 0, 3.0), "e4m3": (torch.float8_e4m3fn, oracle.E4M3, 448.0),
        "e5m2": (torch.float8_e5m2, oracle.E5M2, 57344.0)}


class Case:
    """Random pages for each sequence; slots that no row sees hold NaN."""

    def __init__(self, form, rows, H, G, D, fmt, window=0, sinks=0, seed=0, T=None, MB=None, scale=None):
        # rows: decode (dql, [seq_len...]); varlen [(tokens, prefix)...] with gaps before and behind
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.kind, top = KIND[fmt]
        self.form, self.window, self.sinks = form, window, sinks
        if form == "decode":
            self.dql, lens = rows
            self.seq = np.array(lens, dtype=np.int32)
            B, T = len(lens), len(lens) * self.dql
            self.req, self.pos = oracle.rows_decode(lens, self.dql)
            need = [max(0, n) for n in lens]
        else:
            first, rows = rows
            B = len(rows)
            self.cu = np.concatenate([[first], first + np.cumsum([n for n, _ in rows])]).astype(np.int32)
            self.prefix = np.array([p for _, p in rows], dtype=np.int32)
            T = int(self.cu[-1]) if T is None else T
            self.req, self.pos = oracle.rows_varlen(self.cu, self.prefix, T)
            need = [n + p for n, p in rows]
        MB = MB or max(1, -(-max(need + [1]) // 128))
        pages = B * MB * 8 + 8
        self.table = torch.randperm(B * MB, generator=g).view(B, MB).to(torch.int32)
        self.q = torch.randn((T, H, G, D), generator=g).to(torch.bfloat16)
        self.scale = scale
        seen = torch.zeros((pages, 16, H), dtype=torch.bool)
        for b in range(B):
            for p in self.pos[self.req == b]:
                j = torch.arange(max(0, min(int(p) + 1, MB * 128)))
                if window:
                    j = j[(j > p - window) | (j < sinks)]
                if j.numel():
                    seen[self.table[b, j // 128].long() * 8 + j % 128 // 16, j % 16] = True
        self.c, self.s = [], []
        for _ in range(2):
            x = torch.randn((pages, 16, H, D), generator=g)
            x[~seen] = float("nan")
            if fmt == "bf16":
                self.c.append(x.to(torch.bfloat16))
                self.s.append(None)
            else:
                self.c.append((x * top / 4.5).clamp(-top, top).to(self.dtype))
                self.s.append(torch.exp2(torch.randint(-2, 2, (pages, H), generator=g).float()) * 4.5 / top)

    def bits(self, x):
        return x.view(torch.int16).numpy().view(np.uint16) if self.kind == 0 else x.view(torch.uint8).numpy()

    def want(self, magnitude=False):
        k, v = (self.bits(x) for x in self.c)
        if magnitude:
            v = v & (0x7FFF if self.kind == 0 else 0x7F)
        ks, vs = (None if s is None else s.numpy() for s in self.s)
        scale = self.q.shape[-1] ** -0.5 if self.scale is None else self.scale
        return oracle.paged_attention(self.q, k, v, self.kind, ks, vs, self.table.numpy(), self.req, self.pos, scale,
                                      self.window, self.sinks)

    def args(self, dev):
        i32 = lambda x: torch.from_numpy(x).to(dev)      # noqa: E731
        rows = (i32(self.seq), self.dql) if self.form == "decode" else (i32(self.cu), i32(self.prefix))
        more = dict(window=self.window or None, sinks=self.sinks, scale=self.scale)
        if self.kind:
            more.update(k_scale=self.s[0].to(dev), v_scale=self.s[1].to(dev))
        fn = bsa.bsa_paged_attention_decode if self.form == "decode" else bsa.bsa_paged_attention_varlen
        return fn, (self.q.to(dev), self.c[0].to(dev), self.c[1].to(dev), self.table.to(dev), *rows), more

    def run(self, dev, **kw):
        fn, args, more = self.args(dev)
        return fn(*args, **{**more, **kw})


def check(case, dev, **kw):
    out = torch.full(case.q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    got = case.run(dev, out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    compare(case, got)
    return got


def compare(case, got):
    g, want, mag = got.double().cpu().numpy(), case.want(), case.want(magnitude=True)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 1e-30
    assert np.isfinite(g).all(), np.argwhere(~np.isfinite(g))[:3]
    bad = np.abs(g - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:3], want[bad][:3], tol[bad][:3], bad.mean())
    assert (g[case.pos < 0] == 0).all()


DECODE = [
    (1, [1], 1, 1, 64), (1, [128], 1, 8, 128), (1, [129, 0, 127, 1000], 2, 4, 64), (3, [2, 3, 4, 500], 1, 5, 128),
    (4, [300, 0, 1, 77, 513], 2, 16, 128), (2, [640, 2], 1, 3, 256), (1, [2100], 3, 7, 16), (1, [900, 901], 1, 64, 128),
    (2, [257, 255], 2, 2, 80), (1, [1500], 1, 11, 192), (8, [30, 700], 1, 20, 48),
]


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("dql,lens,H,G,D", DECODE)
def test_decode_rows(cuda_device, fmt, dql, lens, H, G, D):
    check(Case("decode", (dql, lens), H, G, D, fmt, seed=D + G), cuda_device)


VARLEN = [
    # (rows before the first sequence, [(tokens, prefix)...]), H, G, D, rows in all
    ((0, [(1, 0)]), 1, 1, 64, None), ((0, [(128, 0)]), 1, 1, 128, None), ((3, [(7, 0), (0, 50), (5, 200), (130, 3)]), 2, 3, 64, 160),
    ((0, [(300, 0)]), 1, 2, 128, None), ((0, [(33, 1000), (2, 0), (65, 127), (64, 128)]), 1, 4, 128, 170),
    ((1, [(40, 88), (3, 700)]), 2, 5, 256, 50), ((0, [(129, 255)]), 1, 8, 64, None), ((0, [(17, 400)]), 1, 64, 128, None),
    ((0, [(70, 0), (71, 1)]), 1, 6, 80, 141), ((0, [(9, 300), (0, 0), (0, 9)]), 3, 16, 16, 12), ((5, []), 1, 2, 64, 6),
    ((0, [(50, 513)]), 1, 7, 208, None),
]


@pytest.mark.parametrize("fmt", list(KIND))
@pytest.mark.parametrize("rows,H,G,D,T", VARLEN)
def test_varlen_rows(cuda_device, fmt, rows, H, G, D, T):
    check(Case("varlen", rows, H, G, D, fmt, seed=H + G + D, T=T), cuda_device)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 700), (16, 4), (100, 128), (128, 0), (129, 5), (333, 130), (5000, 3)])
@pytest.mark.parametrize("form,rows,H,G,D", [
    ("decode", (2, [1300, 0, 129, 1, 700]), 2, 3, 64), ("decode", (1, [2500, 40]), 1, 8, 128),
    ("varlen", (1, [(200, 300), (3, 0), (77, 1000)]), 1, 4, 128), ("varlen", (0, [(40, 600), (260, 0)]), 1, 2, 256),
])
def test_windows_and_sinks(cuda_device, fmt, window, sinks, form, rows, H, G, D):
    check(Case(form, rows, H, G, D, fmt, window, sinks, seed=window + sinks), cuda_device)


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("scale", [0.0, -0.25, 0.9])
def test_scales_of_the_scores(cuda_device, fmt, scale):
    check(Case("varlen", (0, [(90, 200), (5, 3)]), 1, 4, 64, fmt, seed=4, scale=scale), cuda_device)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_scores_far_apart(cuda_device, fmt):
    """Rows whose maximum rises again and again, by tens of powers of two: the
    token j's score is about j / 8 (or (n - j) / 8), so few probabilities count."""
    for sign in (1.0, -1.0):
        case = Case("varlen", (0, [(150, 600), (20, 900)]), 1, 4, 64, fmt, seed=5)
        # k = ramp along dimension 0 of every token, q picks it; scores up to 118 are exact in 24 bits
        # up to 2^-13, which the bound's 2^-10 covers
        for b in range(2):
            j = torch.arange(case.table.shape[1] * 128)
            page = case.table[b, j // 128].long() * 8 + j % 128 // 16
            k = case.c[0].float() if fmt == "bf16" else None
            if fmt == "bf16":
                k[page, j % 16, 0, 0] = sign * (j // 8).float()
                case.c[0] = k.to(torch.bfloat16)
            else:
                k = case.c[0].float()
                k[page, j % 16, 0, 0] = sign * (j // 64).float()
                case.c[0] = k.to(case.dtype)
                case.s[0][:] = 8.0
        case.q[..., 1:] = 0
        case.q[..., 0] = 1
        case.scale = 1.0
        check(case, cuda_device)


def test_values_with_scales_far_apart(cuda_device):
    """Pages whose value scales differ by 2^60, and scales that are no powers of two."""
    case = Case("varlen", (0, [(140, 500)]), 2, 3, 64, "e4m3", seed=6)
    g = torch.Generator().manual_seed(7)
    case.s[1] *= torch.exp2(torch.randint(-30, 31, case.s[1].shape, generator=g).float()) * 1.3
    case.s[0] *= 0.7
    check(case, cuda_device)


def test_blocks_outside_the_cache_and_past_the_table(cuda_device):
    """Tokens of no page take no part, rows of only such tokens are zeros, and the status
    word says so."""
    dev = cuda_device
    word = torch.zeros(1, dtype=torch.int32, device=dev)
    bsa.bsa_set_status_word(word)
    try:
        for fmt in KIND:
            case = Case("varlen", (0, [(60, 300), (10, 100), (5, 0)]), 1, 3, 64, fmt, seed=8)
            check(case, dev)
            assert bsa.bsa_read_status() == 0
            case.table[0, 1], case.table[1, 0], case.table[2, 0] = -1, case.c[0].shape[0] // 8, 2**31 - 1
            got = check(case, dev)
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID and (got[70:] == 0).all()
            # four pages of a block inside the cache
            case = Case("decode", (1, [200, 100]), 1, 3, 64, fmt, seed=9)
            pages = case.c[0].shape[0] - 4
            case.c = [x[:pages].contiguous() for x in case.c]
            case.s = [None if s is None else s[:pages].contiguous() for s in case.s]
            last = pages // 8
            for x in case.c:
                x[last * 8:] = torch.ones((), dtype=x.dtype) if fmt == "bf16" else x[:1].float().nan_to_num(1.0).to(x.dtype)
            case.table[1, 0] = last
            check(case, dev)
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_BLOCK_ID
            # positions past the table
            case = Case("varlen", (0, [(100, 200)]), 1, 2, 64, fmt, seed=10, MB=2)
            check(case, dev)
            assert bsa.bsa_read_status() == bsa.BSA_STATUS_BAD_CONTEXT
    finally:
        bsa.bsa_set_status_word(None)


def test_an_empty_cache_and_no_rows(cuda_device):
    dev = cuda_device
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev)      # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)              # noqa: E731
    q = torch.ones((4, 2, 3, 64), dtype=torch.bfloat16, device=dev)
    assert (bsa.bsa_paged_attention_decode(q, z(0, 16, 2, 64), z(0, 16, 2, 64), i(4, 3), i(4) + 5, 1) == 0).all()
    assert (bsa.bsa_paged_attention_decode(q, z(8, 16, 2, 64), z(8, 16, 2, 64), i(4, 0), i(4) + 5, 1) == 0).all()
    assert (bsa.bsa_paged_attention_varlen(q, z(8, 16, 2, 64), z(8, 16, 2, 64), i(0, 3), i(1), i(0)) == 0).all()
    assert bsa.bsa_paged_attention_decode(q[:0], z(8, 16, 2, 64), z(8, 16, 2, 64), i(0, 3), i(0), 1).shape == (0, 2, 3, 64)


def _plain(case, dev):
    """Torch in 64 bits on the GPU, for cases too long for the oracle, and the same on |v|."""
    H, G, D = case.q.shape[1:]
    out, mag = (torch.zeros(case.q.shape, dtype=torch.float64, device=dev) for _ in range(2))
    kv = []
    for x, s in zip(case.c, case.s):
        x = x.double()
        kv.append((x if s is None else x * s.double()[:, None, :, None]).nan_to_num(0.0).to(dev))
    q, pos = case.q.double().to(dev), torch.from_numpy(case.pos).to(dev)
    for b in np.unique(case.req):
        rows = torch.from_numpy(np.nonzero((case.req == b) & (case.pos >= 0))[0]).to(dev)
        for part in rows.split(512):
            if part.numel() == 0:
                continue
            p = pos[part]
            j = torch.arange(min(int(p.max()) + 1, case.table.shape[1] * 128), device=dev)
            seen = j <= p[:, None]
            if case.window:
                seen &= (j > p[:, None] - case.window) | (j < case.sinks)
            page = case.table.to(dev)[int(b)].long()[j // 128] * 8 + j % 128 // 16
            for h in range(H):
                k, v = (x[page, j % 16, h] for x in kv)
                s = torch.einsum("tgd,jd->tgj", q[part, h], k) * D ** -0.5
                w = torch.softmax(torch.where(seen[:, None], s, -torch.inf), -1)
                out[part, h], mag[part, h] = w @ v, w @ v.abs()
    return out, mag


@pytest.mark.parametrize("form,rows,H,G,D,fmt,window,sinks", [
    ("varlen", (2, [(1500, 700), (1, 4000), (333, 0)]), 2, 8, 128, "bf16", 0, 0),
    ("varlen", (0, [(2049, 0)]), 3, 4, 64, "e4m3", 0, 0),
    ("varlen", (0, [(700, 2000), (900, 100)]), 1, 5, 256, "bf16", 0, 0),
    ("varlen", (0, [(600, 9000)]), 2, 8, 128, "e5m2", 0, 0),
    ("varlen", (0, [(2500, 1000)]), 2, 8, 128, "bf16", 300, 70),
    ("varlen", (0, [(900, 3000), (800, 0)]), 1, 6, 256, "e4m3", 1000, 10),
    ("decode", (1, [30000, 129, 9000, 1]), 2, 8, 128, "bf16", 0, 0),
    ("decode", (4, [70000]), 1, 16, 128, "e4m3", 0, 0),
    ("decode", (2, [9000 + 77 * i for i in range(80)]), 1, 4, 64, "e4m3", 0, 0),
    ("decode", (1, [12000 + 991 * i for i in range(20)]), 2, 3, 256, "e5m2", 0, 0),
    ("decode", (1, [50000 + 7 * i for i in range(40)]), 2, 8, 128, "bf16", 4096, 4),
])
def test_long_rows(cuda_device, form, rows, H, G, D, fmt, window, sinks):
    """Many items, items split over CTAs, several heads a CTA."""
    case = Case(form, rows, H, G, D, fmt, window, sinks, seed=20)
    got = case.run(cuda_device).double()
    want, mag = _plain(case, cuda_device)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 1e-30
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > tol
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad][:4], float(bad.double().mean()))


@pytest.mark.parametrize("fmt,form,H,G,D", [("bf16", "decode", 2, 4, 64), ("e4m3", "decode", 1, 8, 128), ("bf16", "varlen", 1, 3, 128),
                                            ("e5m2", "varlen", 2, 2, 64), ("bf16", "decode", 1, 2, 256)])
def test_many_sequences(cuda_device, fmt, form, H, G, D):
    """More sequences than a CTA counts at a time, empty ones among them, first and last too."""
    rng = np.random.default_rng(31)
    if form == "decode":
        lens = rng.integers(0, 300, 1300)
        lens[:600] *= rng.integers(0, 2, 600)
        lens[-3:] = 0
        case = Case("decode", (1, lens.tolist()), H, G, D, fmt, seed=31)
    else:
        rows = [(int(n), int(p)) for n, p in zip(rng.integers(0, 4, 1100), rng.integers(0, 260, 1100))]
        rows[:520] = [(0, 5)] * 520
        rows[700] = (150, 40)
        case = Case("varlen", (2, rows), H, G, D, fmt, seed=32)
    got = case.run(cuda_device).double()
    want, mag = _plain(case, cuda_device)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag + 1e-30
    assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all()
    assert (got[torch.from_numpy(case.pos < 0).to(got.device)] == 0).all()


@pytest.mark.parametrize("fmt", list(KIND))
def test_same_bits_again_in_a_graph_and_on_a_side_stream(cuda_device, fmt):
    """A call's bits do not depend on what else runs: again, captured and replayed
    with new lengths, on another stream."""
    dev = cuda_device
    case = Case("decode", (2, [5000, 300, 0, 7777]), 2, 5, 128, fmt, seed=30)
    case.c = [x.float().nan_to_num(0.25).to(x.dtype) for x in case.c]       # slots that later lengths reach
    fn, args, more = case.args(dev)
    ref = fn(*args, **more)
    assert all(torch.equal(fn(*args, **more), ref) for _ in range(3))
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(ref)
    seq = args[4].clone()
    with torch.cuda.graph(graph):
        fn(*args[:4], seq, args[5], out=out, **more)
    side = torch.cuda.Stream(dev)
    for lens in ([5000, 300, 0, 7777], [1, 2, 256, 7000]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            other = fn(*args[:4], seq, args[5], **more)
        torch.cuda.synchronize()
        assert torch.equal(out, other)
    seq.copy_(args[4])
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_offsets_past_32_bits(cuda_device):
    """A cache of more than 2^32 elements: blocks near its end."""
    dev = cuda_device
    H, D, pages = 8, 256, 140000                       # 4.6e9 elements a cache
    blocks = pages // 8
    k, v = (torch.empty((pages, 16, H, D), dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    table = torch.tensor([[blocks - 1, 0], [blocks - 2, blocks // 2 + 1]], dtype=torch.int32)
    ks, vs = torch.ones((pages, H)), torch.ones((pages, H))
    small = Case("decode", (1, [200, 256]), H, 2, D, "e4m3", seed=3)
    for i, x in enumerate((k, v)):
        for b in range(2):
            for n in range(2):
                src = small.table[b, n].long() * 8
                dst = int(table[b, n]) * 8
                x.view(torch.uint8)[dst:dst + 8] = small.c[i].view(torch.uint8)[src:src + 8].to(dev)
                (ks, vs)[i][dst:dst + 8] = small.s[i][src:src + 8]
    fn, args, more = small.args(dev)
    ref = fn(*args, **more)
    more.update(k_scale=ks.to(dev), v_scale=vs.to(dev))
    got = fn(args[0], k, v, table.to(dev), *args[4:], **more)
    assert torch.equal(got, ref)
    del g


def test_refusals(cuda_device):
    dev = cuda_device
    fn, args, more = Case("decode", (1, [100, 50]), 2, 4, 64, "e4m3", seed=1).args(dev)
    q, k, v, table, seq, dql = args
    ok = fn(*args, **more)
    for bad in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(out=q), dict(out=ok[:1]), dict(out=ok.float()),
                dict(out=torch.empty_like(ok, device="cpu")), dict(k_scale=None), dict(workspace=torch.empty(8))):
        with pytest.raises(ValueError):
            fn(*args, **{**more, **bad})
    for bad in ((q.float(), k, v, table, seq, 1), (q, k.float(), v, table, seq, 1), (q, k, v[:-1], table, seq, 1),
                (q, k, v, table.long(), seq, 1), (q, k, v, table[:1], seq, 1), (q, k, v, table, seq.cpu(), 1),
                (q.transpose(0, 1), k, v, table, seq, 1), (q, k, v, None, seq, 1)):
        with pytest.raises(ValueError):
            fn(*bad, **more)
    with pytest.raises(bsa.BsaError) as e:
        fn(q, k, v, table, seq, 2, **more)
    assert e.value.status == -6
    with pytest.raises(ValueError):
        bsa.bsa_paged_attention_varlen(q, k, v, table, [0, 1, 2], seq, **more)
    with pytest.raises(ValueError):
        bsa.bsa_paged_attention_varlen(q, k, v, table, seq, seq, **more)
