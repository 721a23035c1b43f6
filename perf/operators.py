"""Measured cases of the serving operators around the sparse block table.

Three operators that a decode or prefill step runs around the selector:

- ``rope``: rotary positions with several axes (text, or time / height /
  width), forward and inverse (the inverse is the backward pass);
- ``append``: the step's keys, rotated, and values into the paged cache, in
  bf16 or in 8 bits with one scale per 16-token page and head, with the
  step's queries rotated in the same call;
- ``attend``: attention of each row's query heads over its page-16 sparse
  context, read from the 8-bit cache.

``run`` computes them with elementary torch operations, or with this
repository's entry points where ``own`` is true.
"""
import math

import torch

own = False

PAGE = 16
BLOCK = 128
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


def _device():
    return torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request decoding alone: the call's latency
        {"name": "attend one token", "op": "attend", "B": 1, "dql": 1, "H": 1, "G": 8, "D": 128, "K": 16,
         "MB": 74, "lo": 9000, "hi": 9400, "fmt": "e4m3"},
        # the production decode graph: 64 requests, query length 4, 74 blocks, topk 16
        {"name": "attend production", "op": "attend", "B": 64, "dql": 4, "H": 4, "G": 4, "D": 64, "K": 16,
         "MB": 74, "lo": 1, "hi": 9472, "fmt": "e4m3"},
        # long-context decode: 128 requests of up to 131072 tokens, topk 64
        {"name": "attend long topk 64", "op": "attend", "B": 128, "dql": 1, "H": 2, "G": 8, "D": 128, "K": 64,
         "MB": 1024, "lo": 16384, "hi": 131072, "fmt": "e4m3"},
        # few requests that attend to everything: the longest rows a table holds
        {"name": "attend few, whole context", "op": "attend", "B": 3, "dql": 1, "H": 2, "G": 16, "D": 128, "K": 1024,
         "MB": 1024, "lo": 100000, "hi": 131072, "fmt": "e4m3"},
        # wide heads, an odd group, ragged lengths, the other 8-bit type
        {"name": "attend wide ragged", "op": "attend", "B": 37, "dql": 3, "H": 1, "G": 5, "D": 256, "K": 17,
         "MB": 96, "lo": 0, "hi": 12000, "fmt": "e5m2"},
        # one token of one request into the 8-bit cache: the call's latency
        {"name": "append one token", "op": "append", "form": "decode", "B": 1, "dql": 1, "H": 1, "G": 8, "D": 128,
         "MB": 74, "lo": 9000, "hi": 9400, "fmt": "e4m3", "rot": 128, "axes": 1, "pairs": "half"},
        # the production decode graph's step into the 8-bit cache
        {"name": "append production", "op": "append", "form": "decode", "B": 64, "dql": 4, "H": 4, "G": 4, "D": 64,
         "MB": 74, "lo": 1, "hi": 9472, "fmt": "e4m3", "rot": 32, "axes": 1, "pairs": "half"},
        # two prompts of 8192 tokens into the 8-bit cache
        {"name": "append two prompts", "op": "append", "form": "varlen", "B": 2, "L": 8192, "H": 4, "G": 8, "D": 128,
         "MB": 128, "lo": 0, "hi": 8000, "fmt": "e4m3", "rot": 64, "axes": 1, "pairs": "half"},
        # ragged prompts with image positions into the bf16 cache
        {"name": "append ragged, 3 axes, bf16", "op": "append", "form": "varlen", "B": 11, "L": 777, "H": 2, "G": 8,
         "D": 128, "MB": 64, "lo": 0, "hi": 5000, "fmt": "bf16", "rot": 128, "axes": 3, "pairs": "half"},
        # one small image
        {"name": "rope image", "op": "rope", "T": 1369, "H": 16, "D": 64, "rot": 64, "axes": 2, "dtype": "bf16",
         "pairs": "half", "inverse": False},
        # a video clip, time / height / width, in a fused query-key-value buffer
        {"name": "rope video", "op": "rope", "T": 32760, "H": 24, "D": 128, "rot": 128, "axes": 3, "dtype": "bf16",
         "pairs": "interleaved", "inverse": False},
        # the gradient of long text rows in fp32, part of the head rotated
        {"name": "rope backward fp32", "op": "rope", "T": 16411, "H": 10, "D": 128, "rot": 64, "axes": 1,
         "dtype": "fp32", "pairs": "half", "inverse": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "rope"])
    if op == "rope":
        D = rng.choice([32, 64, 80, 128, 256])
        H = rng.randint(1, 24)
        return {"op": op, "T": _log(rng, 1, 1 + 90_000_000 // (H * D)), "H": H, "D": D,
                "rot": 2 * rng.randint(1, D // 2), "axes": rng.randint(1, 4), "dtype": rng.choice(["bf16", "fp32"]),
                "pairs": rng.choice(["half", "interleaved"]), "inverse": rng.random() < 0.5}
    D = rng.choice([64, 128, 256])
    H, G = rng.randint(1, 4), rng.randint(1, 16)
    MB = _log(rng, 8, 1024)
    hi = rng.randint(BLOCK * MB // 2, BLOCK * MB)
    if op == "append":
        case = {"op": op, "H": H, "G": min(G, 8), "D": D, "fmt": rng.choice(["bf16", "e4m3", "e4m3", "e5m2"]),
                "rot": 2 * rng.randint(0, D // 2), "axes": rng.randint(1, 3), "pairs": rng.choice(["half", "interleaved"])}
        if rng.random() < 0.5:
            return {**case, "form": "decode", "B": _log(rng, 1, 512), "dql": rng.randint(1, 4), "MB": min(MB, 128),
                    "lo": 0, "hi": min(hi, BLOCK * min(MB, 128))}
        L = _log(rng, 5, 4000)
        return {**case, "form": "varlen", "B": _log(rng, 1, max(1, min(64, 16384 // L))), "L": L, "MB": L // BLOCK + 40,
                "lo": 0, "hi": 5000}
    K = min(MB, rng.choice([1, 4, 16, 16, 17, 32, 64, 64, 200, 1024]))
    rows = max(1, 2_000_000_000 // (K * BLOCK * D * 8 * H))
    dql = rng.randint(1, 4)
    return {"op": op, "B": _log(rng, 1, max(1, min(128, rows // dql, 130_000 // MB))), "dql": dql, "H": H, "G": G, "D": D, "K": K,
            "MB": MB, "lo": rng.choice([0, hi // 8, hi // 2]), "hi": hi, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(case, dev):
    """theta_i = base^(-2 i / rot) and the axis each frequency turns with, in
    contiguous sections as image models lay them out."""
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    inv = (1_000_000.0 ** (-2.0 * i / max(case["rot"], 1))).to(torch.float32).to(dev)
    axis = (torch.arange(half) * case["axes"] // max(half, 1)).to(torch.int32).to(dev)
    return inv, axis


def _positions(case, T, g, dev):
    """int32 [axes, T]: time / height / width of a grid of patches."""
    side = max(1, int(round(T ** 0.5 / 3)))
    t = torch.arange(T, device=dev)
    rows = [t // (side * side), t // side % side, t % side, t][-case["axes"]:] if case["axes"] > 1 else [t + 100_000]
    start = torch.randint(0, 60_000, (case["axes"], 1), generator=g, device=dev)
    return (torch.stack(rows) + start).to(torch.int32)


def _codes(shape, fmt, g, dev):
    """Cached values as a step leaves them: up to the type's range within a page."""
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)
    if fmt == "bf16":
        return x
    top = F8_MAX[fmt]
    return (x * (top / 4.5)).clamp_(-top, top).to(F8[fmt])


def _page_scales(pages, H, fmt, g, dev):
    s = torch.randint(-1, 2, (pages, H), generator=g, device=dev).to(torch.float32)
    return torch.exp2(s + (-7.0 if fmt == "e4m3" else -14.0))


def _tables(B, MB, g, dev):
    return torch.randperm(B * MB, generator=g, device=dev).to(torch.int32).view(B, MB)


def _sparse_rows(case, table, seq, g, dev):
    """Rows as the selector and its table expansion leave them: the first and
    the own block and random ones between, ascending."""
    B, dql, H, K, MB = case["B"], case["dql"], case["H"], case["K"], case["MB"]
    T = B * dql
    req = torch.arange(T, device=dev) // dql
    length = (seq[req].long() - dql + torch.arange(T, device=dev) % dql + 1).clamp_min(0)
    n = (length + BLOCK - 1) // BLOCK
    b = torch.arange(MB, device=dev)
    r = torch.rand((T, H, MB), generator=g, device=dev)
    r = torch.where((b == 0) | (b == n[:, None, None] - 1), 2.0, r)
    r = torch.where(b < n[:, None, None], r, -1.0)
    top = r.topk(K, dim=2)
    ids = torch.where(top.values >= 0, top.indices, MB).sort(dim=2).values
    kept = ids < MB
    phys = table.long()[req[:, None, None], ids.clamp_max(MB - 1)]
    p = torch.arange(BLOCK // PAGE, device=dev)
    used = kept[..., None] & (ids[..., None] * BLOCK + p * PAGE < length[:, None, None, None])
    bt = torch.where(used, phys[..., None] * (BLOCK // PAGE) + p, 0)
    ctx = (torch.where(kept, length[:, None, None] - ids * BLOCK, 0).clamp(0, BLOCK)).sum(2)
    return bt.reshape(T, H, K * (BLOCK // PAGE)).to(torch.int32).contiguous(), ctx.to(torch.int32).contiguous()


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # heads H of a wider projection output, as a fused query-key-value
        # buffer gives them
        s["x"] = torch.randn((T, H + 2, D), generator=g, device=dev, dtype=dt)[:, 1:1 + H]
        s["inv_freq"], s["freq_axis"] = _frequencies(case, dev)
        s["positions"] = _positions(case, T, g, dev)
        s["out"] = torch.empty((T, H, D), device=dev, dtype=dt)
        return s
    B, H, G, D, MB, fmt = (case[k] for k in ("B", "H", "G", "D", "MB", "fmt"))
    pages = B * MB * (BLOCK // PAGE)
    table = _tables(B, MB, g, dev)
    s["k_cache"] = _codes((pages, PAGE, H, D), fmt, g, dev)
    s["v_cache"] = _codes((pages, PAGE, H, D), fmt, g, dev)
    s["k_scale"] = s["v_scale"] = None
    if fmt != "bf16":
        s["k_scale"] = _page_scales(pages, H, fmt, g, dev)
        s["v_scale"] = _page_scales(pages, H, fmt, g, dev)
    if op == "attend":
        seq = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["bt"], s["ctx"] = _sparse_rows(case, table, seq, g, dev)
        s["q"] = torch.randn((B * case["dql"], H, G, D), generator=g, device=dev, dtype=torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        return s
    s["block_table"] = table
    if case["form"] == "decode":
        T = B * case["dql"]
        s["seq_lens"] = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device=dev).to(torch.int32)
    else:
        lens = torch.randint(max(1, case["L"] - case["L"] // 3), case["L"] + 1, (B,), generator=g, device=dev)
        lens[-1] = B * case["L"] - case["L"] // 5 - lens[:-1].sum() if B > 1 else case["L"]
        lens = lens.clamp(1, MB * BLOCK - 1)
        room = MB * BLOCK - int(lens.max())
        s["prefix_lens"] = torch.randint(case["lo"], min(case["hi"], room) + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["cu_seqlens_q"] = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), lens.cumsum(0)]).to(torch.int32)
        # a token count of its own for the case, with unowned rows at the end
        T = max(B * case["L"], int(lens.sum()))
    qkv = torch.randn((T, (G + 2) * H, D), generator=g, device=dev, dtype=torch.bfloat16)
    s["q"], s["k"], s["v"] = qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]
    s["inv_freq"], s["freq_axis"] = _frequencies(case, dev)
    s["positions"] = _positions(case, T, g, dev) if case["axes"] > 1 else None
    s["q_out"] = torch.empty((T, G * H, D), device=dev, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _rotate(x, positions, inv_freq, freq_axis, pairs, inverse=False):
    """x [T, H, D] in 32 bits, rotated; the angles are taken in 64 bits, where
    far positions keep their fraction of a turn."""
    half = inv_freq.shape[0]
    if half == 0:
        return x.float()
    pos = positions.double()[freq_axis.long()].t()          # [T, half]
    angle = pos * inv_freq.double()
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        sn = -sn
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if pairs == "half":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * c - b * sn, b * c + a * sn], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * sn, b * c + a * sn], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _run_rope(s):
    c = s["case"]
    y = _rotate(s["x"], s["positions"], s["inv_freq"], s["freq_axis"], c["pairs"], c["inverse"])
    return s["out"].copy_(y)


def _rows(s, T):
    """(sequence of each row, its position or -1)."""
    c = s["case"]
    t = torch.arange(T, device=s["k"].device)
    if c["form"] == "decode":
        req = t // c["dql"]
        return req, s["seq_lens"].long()[req] - c["dql"] + t % c["dql"]
    cu = s["cu_seqlens_q"].long()
    req = torch.searchsorted(cu, t, right=True) - 1
    owned = (req >= 0) & (req < c["B"])
    req = req.clamp(0, c["B"] - 1)
    return req, torch.where(owned, s["prefix_lens"].long()[req] + t - cu[req], -1)


def _power_scale(amax, top):
    """The smallest power of two s >= 2^-126 with amax / s <= top; 0 for amax 0."""
    m, e = torch.frexp(amax)
    tm, te = math.frexp(top)
    s = torch.ldexp(torch.ones_like(m), (e - te + (m > tm).to(e.dtype)).clamp_min(-126))
    return torch.where(amax > 0, s, 0.0)


def _store(x, page, off, lead, first, cache, scale, fmt):
    """Values x [n, H, D] in 32 bits into cache[page, off]; `lead` marks the
    first row of a page in this call and `first` that page's first new slot."""
    if fmt == "bf16":
        cache[page, off] = x.to(torch.bfloat16)
        return
    top = F8_MAX[fmt]
    tok = _power_scale(x.abs().amax(-1), top)                                # [n, H]
    lp, lo = page[lead], first[lead]
    old = torch.where(lo[:, None] > 0, scale[lp], 0.0)
    new = torch.zeros_like(scale).index_copy_(0, lp, old)
    new.index_reduce_(0, page, tok, "amax")
    new = torch.where(new > 0, new, 1.0)
    was = cache.view(torch.uint8)[lp].view(F8[fmt]).float()
    ratio = (old / new[lp])[:, None, :, None]
    again = (was * ratio).to(F8[fmt])
    keep = torch.arange(PAGE, device=x.device)[None, :, None, None] >= lo[:, None, None, None]
    cache.view(torch.uint8)[lp] = torch.where(keep, was.to(F8[fmt]).view(torch.uint8), again.view(torch.uint8))
    code = (x / new[page][..., None]).clamp(-top, top).to(F8[fmt])
    cache.view(torch.uint8)[page, off] = code.view(torch.uint8)
    scale[lp] = new[lp]


def _run_append(s):
    c = s["case"]
    T = s["k"].shape[0]
    req, pos = _rows(s, T)
    place = pos[None] if s["positions"] is None else s["positions"]
    args = place, s["inv_freq"], s["freq_axis"], c["pairs"]
    q = torch.where(pos[:, None, None] >= 0, _rotate(s["q"], *args), 0.0)
    s["q_out"].copy_(q)
    live = pos >= 0
    t = torch.arange(T, device=pos.device)
    begin = torch.where(live & (t > 0) & live.roll(1) & (req.roll(1) == req), 0, 1)
    lead = live & ((begin == 1) | (pos % PAGE == 0))
    first = (pos % PAGE)[torch.cummax(torch.where(lead, t, 0), 0).values]
    page = s["block_table"].long()[req, (pos // BLOCK).clamp_min(0)] * (BLOCK // PAGE) + pos % BLOCK // PAGE
    at = (page[live], (pos % PAGE)[live], lead[live], first[live])
    _store(_rotate(s["k"], *args)[live], *at, s["k_cache"], s["k_scale"], c["fmt"])
    _store(s["v"].float()[live], *at, s["v_cache"], s["v_scale"], c["fmt"])
    return _appended(s)


def _appended(s):
    return [s["q_out"], s["k_cache"], s["v_cache"]] + ([] if s["k_scale"] is None else [s["k_scale"], s["v_scale"]])


def _gather(cache, scale, page, h, dtype):
    codes = cache.view(torch.uint8).permute(0, 2, 1, 3)[page, h].view(cache.dtype)      # [T, H, W, 16, D]
    x = codes.to(dtype) * scale.to(dtype)[page, h][..., None, None]
    return x.flatten(2, 3)


def _run_attend(s):
    q, bt, ctx = s["q"], s["bt"].long(), s["ctx"].long()
    T, H, G, D = q.shape
    h = torch.arange(H, device=q.device)[None, :, None]
    live = torch.arange(bt.shape[2] * PAGE, device=q.device) < ctx[..., None]           # [T, H, N]
    k = _gather(s["k_cache"], s["k_scale"], bt, h, torch.float32)
    x = torch.matmul(q.float(), k.transpose(2, 3)) * D ** -0.5
    del k
    x = torch.where(live[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    v = torch.where(live[..., None], _gather(s["v_cache"], s["v_scale"], bt, h, torch.float32), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return s["out"].copy_(o)


def run(state):
    s = state
    if own:
        return _run_own(s)
    return {"rope": _run_rope, "append": _run_append, "attend": _run_attend}[s["op"]](s)


def _run_own(s):
    import block_sparse_attention_topk_gb300 as bsa
    c = s["case"]
    if s["op"] == "rope":
        return bsa.bsa_rope(s["x"], s["positions"], s["inv_freq"], s["freq_axis"], interleaved=c["pairs"] == "interleaved",
                            inverse=c["inverse"], out=s["out"])
    if s["op"] == "attend":
        return bsa.bsa_sparse_decode_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                  s["bt"], s["ctx"], out=s["out"])
    more = dict(q=s["q"], inv_freq=s["inv_freq"], positions=s["positions"], freq_axis=s["freq_axis"],
                interleaved=c["pairs"] == "interleaved", k_scale=s["k_scale"], v_scale=s["v_scale"], q_out=s["q_out"])
    if c["form"] == "decode":
        bsa.bsa_append_kv_decode(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], c["dql"], **more)
    else:
        bsa.bsa_append_kv_varlen(s["k"], s["v"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens_q"],
                                 s["prefix_lens"], **more)
    return _appended(s)


# ---------------------------------------------------------------------------
# bytes and operations
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * n * size + 4 * c["axes"] * c["T"], "flops": 3 * c["T"] * c["H"] * c["rot"]}
    size = 2 if c["fmt"] == "bf16" else 1
    row = c["H"] * c["D"]
    if c["op"] == "append":
        T = c["B"] * (c["dql"] if c["form"] == "decode" else c["L"])
        scales = 0 if c["fmt"] == "bf16" else 8 * c["H"] * (T if c["form"] == "decode" else T // PAGE)
        return {"bytes": T * row * (4 * c["G"] + 4 + 2 * size) + scales + 4 * T, "flops": 3 * T * c["H"] * (c["G"] + 1) * c["rot"]}
    rows = c["B"] * c["dql"] * c["H"]
    mean = (c["lo"] + c["hi"]) / 2
    ctx = min(mean, c["K"] * BLOCK)
    tokens = min(rows * ctx, c["B"] * c["H"] * mean)           # rows of one request share blocks
    return {"bytes": tokens * (2 * c["D"] + 0.5) + rows * (4 * c["G"] * c["D"] + ctx / 4), "flops": 4 * rows * ctx * c["G"] * c["D"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _turned(x, angle, pairs, sign):
    """Complex rotation: a pair (a, b) times e^(i sign angle)."""
    x = x.double()
    half = angle.shape[1]
    z = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    y = x.clone()
    first = slice(0, half) if pairs == "half" else slice(0, 2 * half, 2)
    second = slice(half, 2 * half) if pairs == "half" else slice(1, 2 * half, 2)
    w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _angles(place, s):
    return torch.stack([place[int(a)].double() * f for a, f in zip(s["freq_axis"].tolist(), s["inv_freq"].double())], 1) \
        if s["inv_freq"].numel() else place.new_zeros((place.shape[1], 0), dtype=torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _turned(s["x"], _angles(s["positions"], s), c["pairs"], -1.0 if c["inverse"] else 1.0)
    if c["op"] == "attend":
        q, bt, ctx = s["q"].double(), s["bt"], s["ctx"].tolist()
        T, H, G, D = q.shape
        if T * H > 4096:
            return None
        out = torch.zeros_like(q)
        for t in range(T):
            for h in range(H):
                n = ctx[t][h]
                if n > 0:
                    pages = bt[t, h, :(n + PAGE - 1) // PAGE].long()
                    k, v = (((x[:, :, h].view(torch.uint8)[pages].view(x.dtype).double() * sc[pages, h, None, None].double())
                             .reshape(-1, D)[:n]) for x, sc in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
                    out[t, h] = torch.softmax(q[t, h] @ k.t() / math.sqrt(D), -1) @ v
        return out
    # append: page by page on the host
    T = s["k"].shape[0]
    if c["form"] == "decode":
        seq = s["seq_lens"].tolist()
        owner = [(t // c["dql"], seq[t // c["dql"]] - c["dql"] + t % c["dql"]) for t in range(T)]
    else:
        cu, pre = s["cu_seqlens_q"].tolist(), s["prefix_lens"].tolist()
        owner = [(i, pre[i] + j) for i in range(c["B"]) for j in range(cu[i + 1] - cu[i])]
        owner = [(0, -1)] * cu[0] + owner
        owner += [(0, -1)] * (T - len(owner))
    pos = torch.tensor([p for _, p in owner], device=s["k"].device)
    place = pos[None] if s["positions"] is None else s["positions"]
    angle = _angles(place, s)
    q = _turned(s["q"], angle, c["pairs"], 1.0) * (pos >= 0).double()[:, None, None]
    table = s["block_table"].tolist()
    pages = {}
    for t, (r, p) in enumerate(owner):
        if p >= 0:
            pages.setdefault(table[r][p // BLOCK] * 8 + p % BLOCK // PAGE, []).append((t, p % PAGE))
    ids = list(pages)
    # rows of each page, padded to 16 with row T (zeros)
    rows = torch.full((len(ids), PAGE), T)
    low = torch.tensor([min(o for _, o in pages[i]) for i in ids], dtype=torch.long)
    flat = [(n, o, t) for n, i in enumerate(ids) for t, o in pages[i]]
    if flat:
        n, o, t = torch.tensor(flat).t()
        rows[n, o] = t
    dev = s["k"].device
    rows, low, at = rows.to(dev), low.to(dev), torch.tensor(ids, dtype=torch.long, device=dev)
    outs, scales = [], []
    for x, cache, scale in ((_turned(s["k"], angle, c["pairs"], 1.0), s["k_cache"], s["k_scale"]),
                            (s["v"].double(), s["v_cache"], s["v_scale"])):
        x = torch.cat([x, torch.zeros_like(x[:1])])[rows]                    # [pages, 16, H, D]
        new = (rows < T)[:, :, None, None]
        whole = cache.to(torch.float64)
        if scale is None:
            whole[at] = torch.where(new, x, whole[at])
        else:
            old = torch.where(low[:, None] > 0, scale[at].double(), 0.0)
            need = x.abs().amax((1, 3)) / F8_MAX[c["fmt"]]
            power = torch.where(need > 0, torch.exp2(torch.ceil(torch.log2(need))), 0.0)
            now = torch.maximum(old, power)
            now = torch.where(now > 0, now, 1.0)
            before = torch.arange(PAGE, device=dev)[None, :, None, None] < low[:, None, None, None]
            was = whole[at]
            was = torch.where(before, was * (old / now)[:, None, :, None], was)
            whole[at] = torch.where(new, x / now[:, None, :, None], was)
            sc = scale.double()
            sc[at] = now
            scales.append(sc)
        outs.append(whole)
    return [q] + outs + scales
