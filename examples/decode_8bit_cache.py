"""A sparse decode loop over an 8-bit key/value cache, end to end.

Two requests' prompts go into the paged cache (keys rotated at time / height /
width positions, both in e4m3 with a scale per page and head); then each step
appends one token per request, scores and selects 128-token blocks, expands
them into the page-16 table, and attends to them in the 8-bit cache:

    bsa_append_kv_varlen -> [ bsa_append_kv_decode -> bsa_index_score_topk_select
    -> bsa_sparse_decode_attention_q8 ] x steps

The same tokens also go into a bf16 cache read by bsa_sparse_decode_attention;
the relative difference of the two outputs, the cache's rounding, is printed.

    python examples/decode_8bit_cache.py [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_sparse_attention_topk_gb300 as bsa  # noqa: E402


def run(steps: int = 8, prompts=(5000, 3217), H: int = 2, G: int = 8, D: int = 128, K: int = 16,
        seed: int = 0, device="cuda:0"):
    """Returns the outputs of every step, [(8-bit bf16, bf16-cache fp32)]."""
    dev = torch.device(device)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B = len(prompts)
    blocks = [-(-(p + steps) // bsa.PAGE_SIZE) for p in prompts]
    MB = max(blocks + [K])
    phys = torch.randperm(B * MB, generator=g, device=dev)
    table = phys.to(torch.int32).view(B, MB)
    pages = B * MB * bsa.PAGES_PER_SPARSE_BLOCK
    shape = (pages, 16, H, D)
    kc8, vc8 = (torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
    ks, vs = (torch.ones((pages, H), device=dev) for _ in range(2))
    kc16, vc16 = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))
    index_keys = torch.zeros((B * MB, 64), dtype=torch.bfloat16, device=dev)
    index_keys.normal_(generator=g)
    # three position axes in sections, as for images among text
    half = D // 2
    inv_freq = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(dev)
    axis = (torch.arange(half) * 3 // half).to(torch.int32).to(dev)

    def tokens(T):
        qkv = torch.randn((T, (G + 2) * H, D), generator=g, device=dev).to(torch.bfloat16)
        return qkv[:, :G * H], qkv[:, G * H:(G + 1) * H], qkv[:, (G + 1) * H:]

    def places(pos):
        """int32 [3, T]: text positions, or a 64-wide grid of patches in the first 1024."""
        image = pos < 1024
        return torch.stack([torch.where(image, 0, pos), torch.where(image, pos // 64, pos),
                            torch.where(image, pos % 64, pos)]).to(torch.int32).contiguous()

    def append(form, q, k, v, *rows, pos):
        common = dict(q=q, inv_freq=inv_freq, positions=places(pos), freq_axis=axis)
        form(k, v, kc16, vc16, table, *rows, **common)
        return form(k, v, kc8, vc8, table, *rows, k_scale=ks, v_scale=vs, **common)

    lens = torch.tensor(prompts, device=dev)
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)]).to(torch.int32)
    q, k, v = tokens(sum(prompts))
    pos = torch.cat([torch.arange(p, device=dev) for p in prompts])
    append(bsa.bsa_append_kv_varlen, q, k, v, cu, torch.zeros(B, dtype=torch.int32, device=dev),
           pos=pos)
    outs = []
    for step in range(steps):
        seq_lens = (lens + step + 1).to(torch.int32)
        q, k, v = tokens(B)
        q = append(bsa.bsa_append_kv_decode, q, k, v, seq_lens, 1, pos=lens + step)
        q_idx = torch.randn((B, H, 64), generator=g, device=dev).to(torch.bfloat16)
        _, _, bt, ctx = bsa.bsa_index_score_topk_select(q_idx, index_keys, table, seq_lens, 1, K, 1, 1,
                                                        with_table=True)
        q = q.view(B, H, G, D)
        outs.append((bsa.bsa_sparse_decode_attention_q8(q, kc8, vc8, ks, vs, bt, ctx),
                     bsa.bsa_sparse_decode_attention(q, kc16, vc16, bt, ctx)))
    return outs


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    for i, (a, b) in enumerate(run(ap.parse_args().steps)):
        print(f"step {i}: 8-bit against bf16 cache, relative difference "
              f"{float((a.float() - b).norm() / b.norm()):.4f}")
