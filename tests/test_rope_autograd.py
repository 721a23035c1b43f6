"""How bsa_rope joins autograd, without a GPU: the rotation itself is a stand-in
on CPU tensors."""
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa


class Turn:
    """Rotates half-split pairs by positions * inv_freq."""

    def rope(self, x, positions, inv_freq, freq_axis, interleaved, inverse, out):
        assert not torch.is_grad_enabled() or not x.requires_grad
        half = inv_freq.numel()
        a = positions[:, None] * inv_freq * (-1 if inverse else 1)
        c, s = a.cos()[:, None], a.sin()[:, None]
        u, v = x[..., :half], x[..., half:2 * half]
        y = torch.cat([u * c - v * s, v * c + u * s, x[..., 2 * half:]], -1)
        return y if out is None else out.copy_(y)


@pytest.fixture(autouse=True)
def stand_in(monkeypatch):
    monkeypatch.setattr(bsa, "_binding", lambda: Turn())


def test_gradient():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((5, 2, 8), generator=g, dtype=torch.float64, requires_grad=True)
    pos, inv = torch.arange(5), torch.rand(3, generator=g, dtype=torch.float64)
    assert torch.autograd.gradcheck(lambda t: bsa.bsa_rope(t, pos, inv), x)
    assert torch.autograd.gradcheck(lambda t: bsa.bsa_rope(t, pos, inv, inverse=True), x)
    assert torch.autograd.gradgradcheck(lambda t: bsa.bsa_rope(t, pos, inv) ** 2, x)
    bsa.bsa_rope(x, pos, inv).sum().backward()          # an expanded gradient
    assert x.grad is not None


def test_refusals():
    x = torch.randn((5, 2, 8), requires_grad=True)
    pos, inv = torch.arange(5), torch.rand(3)
    with pytest.raises(ValueError, match="out"):
        bsa.bsa_rope(x, pos, inv, out=torch.empty(5, 2, 8))
    with pytest.raises(ValueError, match="out"):
        bsa.bsa_rope(x.detach(), pos, inv, out=x)
    with pytest.raises(ValueError, match="inv_freq"):
        bsa.bsa_rope(x.detach(), pos, inv.requires_grad_())
    with torch.no_grad():
        assert not bsa.bsa_rope(x, pos, inv).requires_grad
        out = torch.empty(5, 2, 8)
        assert bsa.bsa_rope(x, pos, inv, out=out) is out
