"""Prompts in chunks, then beams over one paged cache, end to end on the device.

Each prompt goes into the cache chunk by chunk, every chunk attending to all
that its request holds; then every request is forked into beams, and each step
reorders the beams, makes room for a token, appends it and attends to the whole
cache and, as a windowed layer would, to a window and the first tokens.  Half
way one request is freed and the cache compacted:

    [ bsa_fork_requests -> bsa_append_kv_varlen -> bsa_paged_attention_varlen ] x chunks
    -> [ bsa_fork_requests -> bsa_append_kv_decode -> bsa_paged_attention_decode x 2 ] x steps
       (-> bsa_compact_blocks)

Nothing in between waits for the device: lengths, tables and reference counts
stay there.  The same runs over a bf16 cache and an e4m3 one; the relative
difference of their outputs, the cache's rounding, is printed.

    python examples/beam_decode_paged_cache.py [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_sparse_attention_topk_gb300 as bsa  # noqa: E402

WINDOW, SINKS = 256, 4


class Cache:
    """One layer's keys and values and the state of its blocks."""

    def __init__(self, blocks, max_blocks, H, D, dtype, dev):
        shape = (blocks * bsa.PAGES_PER_SPARSE_BLOCK, 16, H, D)
        self.k, self.v = (torch.empty(shape, dtype=dtype, device=dev) for _ in range(2))
        self.scales = {}
        if dtype != torch.bfloat16:
            self.scales = dict(k_scale=torch.ones(shape[0], H, device=dev), v_scale=torch.ones(shape[0], H, device=dev))
        self.table = torch.zeros((0, max_blocks), dtype=torch.int32, device=dev)
        self.lens = torch.zeros(0, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(blocks, dtype=torch.int32, device=dev)

    def tensors(self):
        return [self.k, self.v, *self.scales.values()]

    def fork(self, parent, new_tokens):
        """parent None: everyone stays, with room for new_tokens."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.refs.device)      # noqa: E731
        parent = torch.arange(len(new_tokens), dtype=torch.int32, device=self.refs.device) if parent is None else i32(parent)
        self.table, self.lens, self.refs = bsa.bsa_fork_requests(self.tensors(), self.table, self.lens, self.refs, parent,
                                                                 i32(new_tokens))

    def compact(self):
        self.table, self.refs, _ = bsa.bsa_compact_blocks(self.tensors(), self.table, self.lens, self.refs)


def run(steps: int = 8, prompts=(700, 331), beams: int = 3, chunk: int = 200, H: int = 2, G: int = 4, D: int = 128,
        seed: int = 0, device="cuda:0", dtypes=(torch.bfloat16, torch.float8_e4m3fn), rotate: bool = True):
    """Returns (outputs, tokens, parents): for each dtype the outputs of every step, [(whole, windowed)]; the appended keys
    and values by step, and the beams' parents by step."""
    dev = torch.device(device)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    B = len(prompts)
    max_blocks = -(-(max(prompts) + steps) // bsa.PAGE_SIZE)
    blocks = B * max_blocks + B * beams * (max_blocks + 2)
    caches = [Cache(blocks, max_blocks, H, D, t, dev) for t in dtypes]
    inv_freq = (1e6 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().to(dev) if rotate else None
    tokens, parents, outputs = [], [], [[] for _ in dtypes]

    def draw(T):
        qkv = torch.randn((T, (G + 2) * H, D), generator=g, device=dev).to(torch.bfloat16)
        return qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]

    def step(cache, q, k, v, rows, form, **more):
        """Appends a step's tokens and attends; rows as the form takes them."""
        append, attend = ((bsa.bsa_append_kv_varlen, bsa.bsa_paged_attention_varlen) if form == "varlen" else
                          (bsa.bsa_append_kv_decode, bsa.bsa_paged_attention_decode))
        turned = append(k, v, cache.k, cache.v, cache.table, *rows, q=q, inv_freq=inv_freq, **cache.scales)
        turned = turned.view(-1, H, G, D)
        return [attend(turned, cache.k, cache.v, cache.table, *rows, **cache.scales, **w)
                for w in ({}, dict(window=WINDOW, sinks=SINKS))]

    # prompts, `chunk` tokens at a time; a request whose prompt is done brings no rows
    done = [0] * B
    while any(d < p for d, p in zip(done, prompts)):
        n = [min(chunk, p - d) for d, p in zip(done, prompts)]
        q, k, v = draw(sum(n))
        cu = torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
        first = not tokens
        for cache, out in zip(caches, outputs):
            before = torch.tensor(done, dtype=torch.int32, device=dev)
            cache.fork([-1] * B if first else None, n)
            out.append(step(cache, q, k, v, (cu, before), "varlen"))
        tokens.append(("prompt", n, q, k, v))
        parents.append(None)
        done = [d + m for d, m in zip(done, n)]
    # beams
    parent = [b for b in range(B) for _ in range(beams)]
    for i in range(steps):
        if i == steps // 2 and B > 1:      # the first request is done: its beams are freed, the cache compacted
            parent = [p for p in parent if p >= beams]
        R = len(parent)
        q, k, v = draw(R)
        for cache, out in zip(caches, outputs):
            cache.fork(parent, [1] * R)
            if i == steps // 2:
                cache.compact()
            out.append(step(cache, q, k, v, (cache.lens, 1), "decode"))
        tokens.append(("step", None, q, k, v))
        parents.append(parent)
        groups = R // beams
        parent = [b * beams + int(torch.randint(0, beams, (1,), generator=host)) for b in range(groups) for _ in range(beams)]
    return outputs, tokens, parents


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    (a, b), _, _ = run(ap.parse_args().steps)
    for i, (x, y) in enumerate(zip(a, b)):
        d = [float((p.float() - q.float()).norm() / p.float().norm()) for p, q in zip(x, y)]
        print(f"pass {i}: 8-bit against bf16 cache, relative difference {d[0]:.4f}, in a window {d[1]:.4f}")
