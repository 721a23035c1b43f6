"""Measured cases of the operators around the whole paged cache.

Four operators that a serving step runs beside the selector and the sparse
attention:

- ``chunk``: attention of new tokens (a chunk of a prompt, or a decode step's
  few) over everything their sequences hold in the paged cache, causal, from
  the bf16 cache or the 8-bit one with a scale per page and head;
- ``window``: the same with a sliding window and a few first tokens that stay
  visible (sinks);
- ``fork``: every request's next state from its parent's: shared blocks, the
  parent's unfinished block copied, room for new tokens, freed requests;
- ``compact``: the blocks in use moved to the lowest ids.

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
INDEX_D = 64      # width of a block's pooled index key


def _device():
    return torch.device("cuda", torch.cuda.current_device())


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request decoding alone in a layer without selection: the call's latency
        {"name": "chunk one token", "op": "chunk", "form": "decode", "B": 1, "L": 1, "H": 1, "G": 8, "D": 128,
         "MB": 74, "lo": 9000, "hi": 9400, "fmt": "bf16", "window": 0, "sinks": 0},
        # the production decode graph: 64 requests, query length 4, 74 blocks, from the 8-bit cache
        {"name": "chunk production decode", "op": "chunk", "form": "decode", "B": 64, "L": 4, "H": 4, "G": 4, "D": 64,
         "MB": 74, "lo": 1, "hi": 9472, "fmt": "e4m3", "window": 0, "sinks": 0},
        # two 8192-token prompts, with and without a cached prefix
        {"name": "chunk two prompts", "op": "chunk", "form": "varlen", "B": 2, "L": 8192, "H": 4, "G": 8, "D": 128,
         "MB": 128, "lo": 0, "hi": 8000, "fmt": "bf16", "window": 0, "sinks": 0},
        # a chunk of a prompt far into a long context, from the 8-bit cache
        {"name": "chunk far into 128k, 8 bits", "op": "chunk", "form": "varlen", "B": 1, "L": 2048, "H": 2, "G": 8,
         "D": 128, "MB": 1024, "lo": 100000, "hi": 129000, "fmt": "e4m3", "window": 0, "sinks": 0},
        # wide heads, an odd group, ragged short chunks, the other 8-bit type
        {"name": "chunk wide ragged", "op": "chunk", "form": "varlen", "B": 7, "L": 333, "H": 1, "G": 5, "D": 256,
         "MB": 96, "lo": 0, "hi": 11900, "fmt": "e5m2", "window": 0, "sinks": 0},
        # long-context decode in a windowed layer: the cost of the window alone
        {"name": "window long decode", "op": "window", "form": "decode", "B": 128, "L": 1, "H": 2, "G": 8, "D": 128,
         "MB": 1024, "lo": 16384, "hi": 131072, "fmt": "bf16", "window": 4096, "sinks": 4},
        # the two prompts in a windowed layer
        {"name": "window two prompts", "op": "window", "form": "varlen", "B": 2, "L": 8192, "H": 4, "G": 8, "D": 128,
         "MB": 128, "lo": 0, "hi": 8000, "fmt": "bf16", "window": 1024, "sinks": 64},
        # ragged short chunks, an odd group, a window that is no whole number of blocks, 8 bits
        {"name": "window ragged, 8 bits", "op": "window", "form": "varlen", "B": 17, "L": 201, "H": 2, "G": 3, "D": 64,
         "MB": 64, "lo": 0, "hi": 7900, "fmt": "e4m3", "window": 333, "sinks": 5},
        # the four beams of one request take one step: the call's latency
        {"name": "fork four beams", "op": "fork", "R": 4, "beams": 4, "shared": 8960, "lo": 9000, "hi": 9400, "H": 1,
         "D": 128, "MB": 80, "fmt": "e4m3", "spare": 64, "freed": 0.0},
        # 128 requests of four beams each, some of them finished
        {"name": "fork 512 beams", "op": "fork", "R": 512, "beams": 4, "shared": 6144, "lo": 6200, "hi": 8100, "H": 4,
         "D": 128, "MB": 74, "fmt": "bf16", "spare": 1024, "freed": 0.05},
        # a small cache with half of its blocks free
        {"name": "compact small", "op": "compact", "R": 8, "beams": 2, "shared": 256, "lo": 0, "hi": 1200, "H": 1,
         "D": 128, "MB": 16, "fmt": "e4m3", "spare": 64},
        # a large one
        {"name": "compact large", "op": "compact", "R": 256, "beams": 1, "shared": 0, "lo": 1000, "hi": 8190, "H": 4,
         "D": 128, "MB": 64, "fmt": "bf16", "spare": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "window", "window", "fork", "compact"])
    fmt = rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
    if op in ("chunk", "window"):
        D = rng.choice([64, 128, 128, 256])
        H, G = rng.randint(1, 4), rng.randint(1, 16)
        MB = _log(rng, 8, 1024)
        # the padded scores of one KV head and the products of all of them
        room = min(1_500_000_000 // G, 2_000_000_000_000 // (4 * D * G * H)) // (MB * BLOCK)
        form = rng.choice(["decode", "varlen"])
        if form == "decode":
            L = rng.randint(1, 4)
            B = _log(rng, 1, max(1, min(256, room // L, 60_000 // MB)))
        else:
            L = _log(rng, 2, max(2, min(8192, room, MB * BLOCK // 2)))
            B = _log(rng, 1, max(1, min(64, room // L, 16384 // L, 60_000 // MB)))
        hi = rng.randint(MB * BLOCK // 4, MB * BLOCK - L)
        case = {"op": op, "form": form, "B": B, "L": L, "H": H, "G": G, "D": D, "MB": MB,
                "lo": rng.choice([0, hi // 8, hi // 2]), "hi": hi, "fmt": fmt, "window": 0, "sinks": 0}
        if op == "window":
            case["window"] = _log(rng, 1, MB * BLOCK // 2)
            case["sinks"] = rng.choice([0, 1, 4, 5, 64, 200])
        return case
    D, H = rng.choice([64, 128, 256]), rng.randint(1, 4)
    beams = rng.choice([1, 2, 3, 4, 8])
    MB = _log(rng, 4, 128)
    hi = rng.randint(BLOCK, MB * BLOCK - 1)
    shared = 0 if beams == 1 else rng.randint(0, hi // BLOCK) * BLOCK
    lo = rng.randint(shared, hi)
    own_blocks = hi // BLOCK + 2 - shared // BLOCK
    R = beams * _log(rng, 1, max(1, 2_000_000_000 // (beams * (own_blocks + shared // BLOCK // beams) * BLOCK * H * D * 2)
                                 if op == "compact" else min(512 // beams, 8000 // (beams * own_blocks))))
    R = max(beams, min(R, 512 // beams * beams))
    case = {"op": op, "R": R, "beams": beams, "shared": shared, "lo": lo, "hi": hi, "H": H, "D": D, "MB": MB, "fmt": fmt,
            "spare": rng.randint(1, 200)}
    if op == "fork":
        case["spare"] += 2 * R
        case["freed"] = rng.choice([0.0, 0.1])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

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


def _blocks_needed(case):
    """Blocks of a fork or compact case's cache: the requests' at most, and the spare ones."""
    groups, s = case["R"] // case["beams"], case["shared"] // BLOCK
    return groups * s + case["R"] * (case["hi"] // BLOCK + 1 - s) + case["spare"]


def _prepare_blocks(case, s, g, dev):
    """Requests in groups that share their first blocks, as forks of one prompt
    do, their blocks scattered over the cache."""
    R, beams, MB = case["R"], case["beams"], case["MB"]
    groups, first = R // beams, case["shared"] // BLOCK
    n = _blocks_needed(case)
    lens = torch.randint(case["lo"], case["hi"] + 1, (R,), generator=g, device=dev)
    held = (lens + BLOCK - 1) // BLOCK
    j = torch.arange(MB, device=dev)
    alone = (j >= first) & (j < held[:, None])
    number = torch.where(alone, groups * first + alone.flatten().cumsum(0).view(R, MB) - 1,
                         torch.arange(R, device=dev)[:, None] // beams * first + j.clamp_max(max(first - 1, 0)))
    ids = torch.randperm(n, generator=g, device=dev)
    table = torch.where(j < held[:, None], ids[number], -1)
    refs = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    refs.index_add_(0, torch.where(table >= 0, table, n).flatten(), torch.ones(R * MB, dtype=torch.int32, device=dev))
    s["block_table"], s["seq_lens"], s["block_refs"] = table.to(torch.int32), lens.to(torch.int32), refs[:n].clone()
    s["k_idx"] = torch.randn((n, INDEX_D), generator=g, device=dev, dtype=torch.bfloat16)
    if case["op"] == "fork":
        r = torch.arange(R, device=dev)
        parent = r // beams * beams + torch.randint(0, beams, (R,), generator=g, device=dev)
        gone = torch.rand(R, generator=g, device=dev) < case["freed"]
        s["parent"] = torch.where(gone, -1, parent).to(torch.int32)
        s["new_tokens"] = torch.where(gone, 0, 1).to(torch.int32)
    return n


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op, H, D, fmt = case["op"], case["H"], case["D"], case["fmt"]
    s = {"case": case, "op": op}
    attends = op in ("chunk", "window")
    blocks = case["B"] * case["MB"] if attends else _prepare_blocks(case, s, g, dev)
    pages = blocks * (BLOCK // PAGE)
    s["k_cache"] = _codes((pages, PAGE, H, D), fmt, g, dev)
    s["v_cache"] = _codes((pages, PAGE, H, D), fmt, g, dev)
    s["k_scale"] = s["v_scale"] = None
    if fmt != "bf16":
        s["k_scale"] = _page_scales(pages, H, fmt, g, dev)
        s["v_scale"] = _page_scales(pages, H, fmt, g, dev)
    if not attends:
        return s
    B, L, MB = case["B"], case["L"], case["MB"]
    s["block_table"] = torch.randperm(blocks, generator=g, device=dev).to(torch.int32).view(B, MB)
    if case["form"] == "decode":
        s["seq_lens"] = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device=dev).to(torch.int32)
    else:
        # chunks of L tokens or somewhat fewer; rows of no sequence at the end
        lens = torch.randint(max(1, L - L // 3), L + 1, (B,), generator=g, device=dev)
        lens[0] = L - L // 5
        s["prefix_lens"] = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=g, device=dev).to(torch.int32)
        s["cu_seqlens_q"] = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), lens.cumsum(0)]).to(torch.int32)
    s["q"] = torch.randn((B * L, H, case["G"], D), generator=g, device=dev, dtype=torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _rows(s):
    """First row, number of rows and first row's position of each sequence."""
    c = s["case"]
    if c["form"] == "decode":
        start = torch.arange(c["B"], device=s["q"].device) * c["L"]
        return start, torch.full_like(start, c["L"]), s["seq_lens"].long() - c["L"]
    cu = s["cu_seqlens_q"].long()
    return cu[:-1], cu[1:] - cu[:-1], s["prefix_lens"].long()


def _context(cache, scale, blocks, h):
    """Head h of the tokens of `blocks` [B, n] in 32 bits: [B, n * 128, D]."""
    D = cache.shape[3]
    x = cache.view(torch.uint8).view(-1, BLOCK, cache.shape[2], D * cache.element_size())[:, :, h][blocks]
    x = x.view(cache.dtype).float()
    if scale is not None:
        x = x * scale[:, h].view(-1, BLOCK // PAGE)[blocks].repeat_interleave(PAGE, -1)[..., None]
    return x.flatten(1, 2)


def _run_attend(s):
    c, q = s["case"], s["q"]
    T, H, G, D = q.shape
    B, L = c["B"], c["L"]
    start, count, pos0 = _rows(s)
    i = torch.arange(L, device=q.device)
    row = (start[:, None] + i).clamp_max(T - 1)                      # [B, L]
    owned = i < count[:, None]
    pos = torch.where(owned, pos0[:, None] + i, -1)
    n = min(c["MB"], (c["hi"] + L + BLOCK - 1) // BLOCK)
    j = torch.arange(n * BLOCK, device=q.device)
    seen = j <= pos[..., None]
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    held = (j <= pos.amax(1, keepdim=True))[..., None]               # [B, N, 1]
    blocks = s["block_table"].long()[:, :n]
    out = torch.zeros_like(q)
    for h in range(H):      # a head at a time: its scores alone take gigabytes
        k = _context(s["k_cache"], s["k_scale"], blocks, h)
        x = torch.matmul(q[:, h][row].float().view(B, L * G, D), k.transpose(1, 2)).view(B, L, G, -1)
        del k
        x = torch.where(seen[:, :, None], x * D ** -0.5, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
        del x
        total = p.sum(-1, keepdim=True)
        v = torch.where(held, _context(s["v_cache"], s["v_scale"], blocks, h), 0.0)
        o = torch.matmul(p.view(B, L * G, -1), v).view(B, L, G, D) / torch.where(total > 0, total, 1.0)
        del p, v
        out[:, h].index_put_((row[owned],), o[owned].to(out.dtype))
    return s["out"].copy_(out)


def _tensors(s):
    """What a block's id stands for: its keys, values, scales and pooled index key."""
    return [s[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale", "k_idx") if s[k] is not None]


def _move(s, src, dst):
    """The contents of blocks src to blocks dst."""
    n = s["block_refs"].shape[0]
    for t in _tensors(s):
        x = t.view(torch.uint8).view(n, -1)
        x[dst] = x[src]


def _run_fork(s):
    c = s["case"]
    old, lens, refs, parent = s["block_table"].long(), s["seq_lens"].long(), s["block_refs"], s["parent"].long()
    n, (R, MB) = refs.shape[0], old.shape
    j = torch.arange(MB, device=old.device)
    r = torch.arange(parent.shape[0], device=old.device)
    p = parent.clamp_min(0)
    base = torch.where(parent >= 0, lens[p], 0)
    new = base + s["new_tokens"].long()
    kept = j < (base[:, None] + BLOCK - 1) // BLOCK
    # a parent's unfinished block goes to its first child, and in copy to the others
    first = torch.full((R,), r.numel(), device=r.device).scatter_reduce(0, p, torch.where(parent >= 0, r, r.numel()), "amin")
    again = (parent >= 0) & (first[p] != r) & (base % BLOCK > 0)
    copied = again[:, None] & (j == base[:, None] // BLOCK)
    was = j < (lens[:, None] + BLOCK - 1) // BLOCK
    got = kept & ~copied
    after = torch.cat([refs, refs.new_zeros(1)])
    after.index_add_(0, torch.where(was, old, n).flatten(), torch.full((R * MB,), -1, dtype=refs.dtype, device=r.device))
    after.index_add_(0, torch.where(got, old[p], n).flatten(), torch.ones(got.numel(), dtype=refs.dtype, device=r.device))
    after = after[:n].clone()
    fresh = copied | (~kept & (j < (new[:, None] + BLOCK - 1) // BLOCK))
    free = (after == 0).cumsum(0)
    ids = torch.searchsorted(free, fresh.flatten().cumsum(0)).view(fresh.shape)
    table = torch.where(fresh, ids, torch.where(got, old[p], -1))
    after.index_fill_(0, table[fresh], 1)
    _move(s, old[p][copied], table[copied])
    return [table.to(torch.int32), new.to(torch.int32), after] + _tensors(s)


def _run_compact(s):
    old, lens, refs = s["block_table"].long(), s["seq_lens"].long(), s["block_refs"]
    n = refs.shape[0]
    b = torch.arange(n, device=old.device)
    live = refs > 0
    top = live.sum()
    src, dst = (live & (b >= top)).nonzero()[:, 0], (~live & (b < top)).nonzero()[:, 0]
    ids = torch.where(live, b, -1)
    ids[src] = dst
    held = torch.arange(old.shape[1], device=old.device) < (lens[:, None] + BLOCK - 1) // BLOCK
    table = torch.where(held, ids[old.clamp_min(0)], -1)
    after = refs.clone()
    after[dst] = refs[src]
    after[src] = 0
    _move(s, src, dst)
    return [table.to(torch.int32), after, ids.to(torch.int32)] + _tensors(s)


def run(state):
    s = state
    if own:
        return _run_own(s)
    return {"chunk": _run_attend, "window": _run_attend, "fork": _run_fork, "compact": _run_compact}[s["op"]](s)


def _run_own(s):
    import block_sparse_attention_topk_gb300 as bsa
    c = s["case"]
    if s["op"] == "fork":
        return list(bsa.bsa_fork_requests(_tensors(s), s["block_table"], s["seq_lens"], s["block_refs"], s["parent"],
                                          s["new_tokens"])) + _tensors(s)
    if s["op"] == "compact":
        return list(bsa.bsa_compact_blocks(_tensors(s), s["block_table"], s["seq_lens"], s["block_refs"])) + _tensors(s)
    more = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
    if c["window"]:
        more.update(window=c["window"], sinks=c["sinks"])
    if c["form"] == "decode":
        return bsa.bsa_paged_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], c["L"],
                                              **more)
    return bsa.bsa_paged_attention_varlen(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["cu_seqlens_q"],
                                          s["prefix_lens"], **more)


# ---------------------------------------------------------------------------
# bytes and operations
# ---------------------------------------------------------------------------

def _pairs(L, pos0, window, sinks):
    """Visible (query, key) pairs of L tokens from position pos0 on, and the keys that any of them sees."""
    def below(n):       # sum of min(p + 1, n) over p < pos0 + L, p >= pos0
        f = lambda x: x * (x + 1) / 2 if x <= n else n * (n + 1) / 2 + (x - n) * n      # noqa: E731
        return f(pos0 + L) - f(pos0)
    if not window:
        return below(pos0 + L), pos0 + L
    return below(window + sinks), min(pos0 + L, window + L - 1 + sinks)


def work(case):
    c = case
    size = 2 if c["fmt"] == "bf16" else 1
    if c["op"] in ("chunk", "window"):
        L = c["L"] if c["form"] == "decode" else c["L"] * 5 / 6
        mean = max(0.0, (c["lo"] + c["hi"]) / 2 - (L if c["form"] == "decode" else 0))
        pairs, keys = _pairs(L, mean, c["window"], c["sinks"])
        token = 2 * c["D"] * size + (0 if size == 2 else 0.5)
        return {"bytes": c["B"] * c["H"] * (keys * token + 4 * L * c["G"] * c["D"]) + c["B"] * keys / 32,
                "flops": 4 * c["B"] * c["H"] * c["G"] * c["D"] * pairs}
    block = BLOCK * c["H"] * (2 * c["D"] * size + (0 if size == 2 else 0.5)) + 2 * INDEX_D
    n = _blocks_needed(c)
    if c["op"] == "fork":
        k = c["beams"]
        moved = c["R"] * (1 - (1 - (1 - 1 / k) ** k)) * (1 - c["freed"])
    else:
        live = c["R"] // c["beams"] * (c["shared"] // BLOCK) + c["R"] * ((c["lo"] + c["hi"]) / 2 - c["shared"]) / BLOCK
        moved = live * (1 - min(1.0, live / n))
    return {"bytes": 2 * moved * block + 8 * c["R"] * c["MB"] + 8 * n, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "fork":
        return _exact_fork(s)
    if c["op"] == "compact":
        return _exact_compact(s)
    if work(c)["flops"] > 4e12:
        return None
    q = s["q"].double()
    T, H, G, D = q.shape
    out = torch.zeros_like(q)
    if c["form"] == "decode":
        spans = [(i * c["L"], c["L"], n - c["L"]) for i, n in enumerate(s["seq_lens"].tolist())]
    else:
        cu, pre = s["cu_seqlens_q"].tolist(), s["prefix_lens"].tolist()
        spans = [(cu[i], cu[i + 1] - cu[i], pre[i]) for i in range(c["B"])]
    for b, (t0, L, p0) in enumerate(spans):
        n = p0 + L
        if n <= 0 or L <= 0:
            continue
        skip = max(0, -p0)          # rows at negative positions are padding
        ids = s["block_table"][b, :(n + BLOCK - 1) // BLOCK].long()
        # one step of queries at a time, and no keys that none of them sees
        for i0 in range(skip, L, 1024):
            i1 = min(L, i0 + 1024)
            p = torch.arange(p0 + i0, p0 + i1, device=q.device)
            j = torch.arange(p0 + i1, device=q.device)
            if c["window"]:
                j = j[(j < c["sinks"]) | (j > p0 + i0 - c["window"])]
            hidden = j[None] > p[:, None]
            if c["window"]:
                hidden |= (j[None] >= c["sinks"]) & (p[:, None] - j[None] >= c["window"])
            for h in range(H):
                page = ids[j // BLOCK] * 8 + j % BLOCK // PAGE
                k, v = (x[:, :, h].view(torch.uint8)[page, j % PAGE].view(x.dtype).double()
                        * (1.0 if sc is None else sc[page, h].double()[:, None])
                        for x, sc in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
                for g in range(G):
                    w = (q[t0 + i0:t0 + i1, h, g] @ k.t()) / math.sqrt(D)
                    w.masked_fill_(hidden, -math.inf)
                    out[t0 + i0:t0 + i1, h, g] = torch.softmax(w, -1) @ v
    return out


def _exact_state(s):
    lens = s["seq_lens"].tolist()
    rows = [row[:-(-n // BLOCK)] for row, n in zip(s["block_table"].tolist(), lens)]
    return rows, lens, s["block_refs"].tolist()


def _exact_tensors(s, moves):
    n = s["block_refs"].shape[0]
    out = [t.clone() for t in _tensors(s)]
    if moves:
        src, dst = torch.tensor(moves, device=s["block_refs"].device).t()
        for x, t in zip(out, _tensors(s)):
            x.view(torch.uint8).view(n, -1).index_copy_(0, dst, t.view(torch.uint8).view(n, -1)[src])
    return out


def _exact_fork(s):
    rows, lens, refs = _exact_state(s)
    parent, new = s["parent"].tolist(), s["new_tokens"].tolist()
    MB = s["block_table"].shape[1]
    for row in rows:
        for b in row:
            refs[b] -= 1
    taken, state = set(), []
    for p, more in zip(parent, new):
        n = lens[p] if p >= 0 else 0
        row = list(rows[p]) if p >= 0 else []
        source = None
        if p >= 0 and n % BLOCK and p in taken:
            source, row[-1] = row[-1], None
        taken.add(p)
        row += [None] * (-(-(n + more) // BLOCK) - len(row))
        for b in row:
            if b is not None:
                refs[b] += 1
        state.append((row, source, n + more))
    free = iter([b for b, k in enumerate(refs) if k == 0])
    moves = []
    for row, source, _ in state:
        for i, b in enumerate(row):
            if b is None:
                row[i] = next(free)
                refs[row[i]] = 1
                if source is not None:
                    moves.append((source, row[i]))
                    source = None
    dev = s["block_refs"].device
    table = torch.tensor([row + [-1] * (MB - len(row)) for row, _, _ in state], dtype=torch.int32, device=dev)
    return [table, torch.tensor([n for _, _, n in state], dtype=torch.int32, device=dev),
            torch.tensor(refs, dtype=torch.int32, device=dev)] + _exact_tensors(s, moves)


def _exact_compact(s):
    rows, _, refs = _exact_state(s)
    MB = s["block_table"].shape[1]
    top = sum(k > 0 for k in refs)
    low = iter([b for b in range(top) if refs[b] == 0])
    ids = [(b if b < top else next(low)) if k > 0 else -1 for b, k in enumerate(refs)]
    after = [0] * len(refs)
    for b, to in enumerate(ids):
        if to >= 0:
            after[to] = refs[b]
    dev = s["block_refs"].device
    table = torch.tensor([[ids[b] for b in row] + [-1] * (MB - len(row)) for row in rows], dtype=torch.int32, device=dev)
    return [table, torch.tensor(after, dtype=torch.int32, device=dev), torch.tensor(ids, dtype=torch.int32, device=dev)] \
        + _exact_tensors(s, [(b, to) for b, to in enumerate(ids) if to >= 0 and to != b])
