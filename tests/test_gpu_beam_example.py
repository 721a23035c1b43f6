"""The beam example: prompts in chunks, forks, appends, attention with and without a
window, a freed request and compaction together, over a bf16 cache and an 8-bit one.

Without rotation the bf16 cache holds the drawn tokens as they are, so each output is
checked against attention over its row's own history, followed through the forks in
plain Python.  Tolerance as in test_gpu_paged_attention.py.  The 8-bit cache against
the bf16 one: 0.037 relative from the codes' rounding (test_gpu_decode_8bit_example.py),
and 2^-9 for the probabilities of each; 0.06 bounds it."""
import pytest
import torch

from examples.beam_decode_paged_cache import SINKS, WINDOW, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,D,prompts,beams,chunk", [(2, 4, 128, (700, 331), 3, 200), (1, 3, 64, (128, 5, 257), 2, 300),
                                                       (2, 2, 256, (90, 300), 4, 64)])
def test_beams_over_one_cache(cuda_device, H, G, D, prompts, beams, chunk):
    (outs,), tokens, parents = run(steps=6, prompts=prompts, beams=beams, chunk=chunk, H=H, G=G, D=D, seed=D,
                                   dtypes=(torch.bfloat16,), rotate=False)
    torch.cuda.synchronize()
    held = [[] for _ in prompts]                       # each row's tokens: (keys, values) [H, D]
    for (kind, n, q, k, v), parent, out in zip(tokens, parents, outs):
        q, k, v = (x.double() for x in (q, k, v))
        if kind == "prompt":
            rows, at = [], 0
            for b, m in enumerate(n):
                for i in range(m):
                    held[b] = held[b] + [(k[at + i], v[at + i])]
                    rows.append(held[b])
                at += m
        else:
            held = [held[p] + [(k[r], v[r])] for r, p in enumerate(parent)]
            rows = held
        # a few rows of a prompt's chunk, all of a step
        for t in (range(len(rows)) if kind == "step" else sorted({0, 1, len(rows) // 2, len(rows) - 1})):
            kk, vv = (torch.stack([x[i] for x in rows[t]]) for i in range(2))
            j = torch.arange(len(rows[t]), device=kk.device)
            for which, seen in enumerate((j >= 0, (j > len(rows[t]) - 1 - WINDOW) | (j < SINKS))):
                for h in range(H):
                    s = q[t].view(H, G, D)[h] @ kk[seen, h].t() * D ** -0.5
                    w = torch.softmax(s, -1)
                    want, mag = w @ vv[seen, h], w @ vv[seen, h].abs()
                    got = out[which][t, h].double()
                    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * 2.0 ** -10) * (1 + 2.0 ** -8) * mag
                    assert ((got - want).abs() <= tol).all(), (kind, t, which, h)


def test_the_8_bit_cache_against_bf16(cuda_device):
    (a, b), _, _ = run(steps=6)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        for p, q in zip(x, y):
            assert torch.isfinite(q).all()
            assert float((p.float() - q.float()).norm() / p.float().norm()) <= 0.06
