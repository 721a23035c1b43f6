"""Rotary positions with one or several axes against the 64-bit oracle.

Tolerance.  A fraction of a turn is a 24-bit float in [-1, 1): its rounding
moves the angle by at most pi 2^-25, sincospi adds at most 2^-23 to a cosine or
sine, and the step's 53-bit rounding moves the angle by 2 pi p 2^-55 or less.
The two products and the sum round by 2^-24 each.  With m the row's largest
magnitude, |error| <= 2 m (pi 2^-25 + 2^-23 + 2 pi p 2^-55 + 3 * 2^-24), and
bf16 outputs round once more by half a step, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
import synth

pytestmark = pytest.mark.gpu


def bound(x, y, far, bf16):
    m = np.abs(x).max(-1, keepdims=True)
    tol = 2 * m * (math.pi * 2.0 ** -25 + 2.0 ** -23 + 2 * math.pi * far * 2.0 ** -55 + 3 * 2.0 ** -24)
    if bf16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y) + 2.0 ** -134
    return tol


def _case(T, H, D, rot, axes, dtype, seed, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g).to(dtype)
    pos = torch.randint(-50, far, (axes, T), generator=g, dtype=torch.int64).to(torch.int32)
    inv = (1e6 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))).float()
    axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    return x, pos, inv, axis


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot,axes", [
    (1, 1, 2, 2, 1), (1, 8, 128, 128, 1), (3, 5, 80, 80, 3), (257, 3, 128, 64, 2), (33, 2, 96, 62, 3),
    (17, 1, 7, 4, 1), (5, 2, 1024, 1024, 8), (4099, 4, 64, 64, 3), (40, 7, 256, 16, 4), (9, 3, 65, 0, 1),
    (130, 16, 128, 128, 3), (65, 1, 24, 20, 2), (2500, 1, 32, 20, 3), (3001, 2, 16, 16, 1),
])
def test_rope(cuda_device, T, H, D, rot, axes, interleaved, dtype):
    x, pos, inv, axis = _case(T, H, D, rot, axes, dtype, T + D + rot)
    dev = cuda_device
    dp, di, da = pos.to(dev), inv.to(dev), axis.to(dev)
    xd = x.to(dev)
    for inverse in (False, True):
        want = oracle.rope(x.double().numpy(), pos.numpy(), inv.numpy(), axis.numpy(), interleaved, inverse)
        got = bsa.bsa_rope(xd, dp, di, da, interleaved=interleaved, inverse=inverse)
        torch.cuda.synchronize()
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound(x.double().numpy(), want, 1 << 20, dtype == torch.bfloat16)).all(), err.max()
        assert torch.equal(got[..., rot:], xd[..., rot:])
    place = xd.clone()
    assert bsa.bsa_rope(place, dp, di, da, interleaved=interleaved, inverse=True, out=place) is place
    torch.cuda.synchronize()
    assert torch.equal(place, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rope_strided_views(cuda_device, dtype, shift):
    """Heads of a fused buffer and head-major outputs, at any element offset;
    what lies between the rows is left alone."""
    T, H, D, rot = 37, 3, 64, 48
    x, pos, inv, axis = _case(T, H, D, rot, 2, dtype, 5)
    dev = cuda_device
    wide = torch.full((T, (H + 2) * D + 5), 9.0, dtype=dtype, device=dev)
    view = wide[:, shift:shift + H * D].unflatten(1, (H, D))
    view.copy_(x.to(dev))
    buf = torch.full((H, T, D + shift), 7.0, dtype=dtype, device=dev)
    out = buf[:, :, shift:].transpose(0, 1)
    bsa.bsa_rope(view, pos.to(dev), inv.to(dev), axis.to(dev), out=out)
    torch.cuda.synchronize()
    want = oracle.rope(x.double().numpy(), pos.numpy(), inv.numpy(), axis.numpy())
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound(x.double().numpy(), want, 1 << 20, dtype == torch.bfloat16)).all()
    assert (buf[:, :, :shift] == 7).all() and (wide[:, shift + H * D:] == 9).all()


def test_rope_far_positions(cuda_device):
    """Positions up to 2^31 - 1 keep their fraction of a turn."""
    x, pos, inv, _ = _case(64, 2, 64, 64, 1, torch.float32, 8)
    pos[0, :8] = torch.tensor([2**31 - 1, -2**31, 2**31 - 2, 10**9, 123456789, 0, -1, 1])
    got = bsa.bsa_rope(x.to(cuda_device), pos[0].to(cuda_device), inv.to(cuda_device))
    torch.cuda.synchronize()
    want = oracle.rope(x.double().numpy(), pos.numpy(), inv.numpy())
    # the oracle's own angle, up to 2^31 rad, is rounded to 2^-23
    tol = bound(x.double().numpy(), want, 2.0 ** 31, False) + 2 * np.abs(x.numpy()).max() * 2.0 ** -22
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(cuda_device, interleaved):
    """The inverse rotation of a gradient is the gradient: against the
    transposed rotation in 64 bits and against differences (exact up to
    rounding, as the map is linear)."""
    T, H, D, rot = 11, 2, 32, 24
    x, pos, inv, axis = _case(T, H, D, rot, 3, torch.float32, 21)
    dy = synth.normal_scores((T, H, D), torch.float32, seed=22)
    dev = cuda_device
    dx = bsa.bsa_rope(dy.to(dev), pos.to(dev), inv.to(dev), axis.to(dev), interleaved=interleaved,
                      inverse=True).double().cpu().numpy()
    args = (pos.numpy(), inv.numpy(), axis.numpy(), interleaved)
    eye = np.broadcast_to(np.eye(D)[:, None, None], (D, T, H, D))
    jac = np.stack([oracle.rope(e, *args) for e in eye])            # [D in, T, H, D out]
    want = np.einsum("ithd,thd->thi", jac, dy.double().numpy())
    tol = bound(dy.double().numpy(), want, 1 << 20, False)
    assert (np.abs(dx - want) <= tol).all()
    step = synth.normal_scores((T, H, D), torch.float32, seed=23).double().numpy()
    base = x.double().numpy()
    diff = ((oracle.rope(base + step, *args) - oracle.rope(base - step, *args)) / 2 * dy.double().numpy()).sum(-1)
    assert np.abs((dx * step).sum(-1) - diff).max() <= D * tol.max() * np.abs(step).max()


def test_rope_special_values_and_streams(cuda_device):
    """NaN and infinities stay within their pair; a side stream; a graph."""
    T, H, D = 6, 2, 16
    x, pos, inv, _ = _case(T, H, D, D, 1, torch.float32, 31)
    x[0, 0, 3], x[1, 1, 9] = float("nan"), float("inf")
    dev = cuda_device
    xd, pd, fd = x.to(dev), pos[0].to(dev), inv.to(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(dev)
    with torch.cuda.stream(s):
        got = bsa.bsa_rope(xd, pd, fd)
    s.synchronize()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[0, 0, [3, 11]] = True
    want[1, 1, [1, 9]] = True
    assert torch.equal(bad, want)
    out = torch.empty_like(xd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bsa.bsa_rope(xd, pd, fd, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.nan_to_num(5, 6, 7), got.nan_to_num(5, 6, 7))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot,offset", [
    (1, 1, 8, 8, 0), (301, 3, 72, 72, 0), (37, 5, 72, 64, 4), (33, 2, 80, 72, 4), (9, 4, 136, 40, 0),
    (2050, 2, 64, 24, 4), (5, 1, 1016, 1016, 4), (65, 3, 128, 104, 0), (12, 2, 88, 0, 4), (12, 2, 72, 62, 4),
])
def test_rope_rows_at_multiples_of_8_bytes(cuda_device, T, H, D, rot, offset, interleaved):
    """bf16 rows that start at odd multiples of 8 bytes, or pairs whose distance
    is one: out of place, and in place with the same bits."""
    x, pos, inv, axis = _case(T, H, D, rot, 2, torch.bfloat16, T + D + rot + offset)
    dev = cuda_device
    fused = torch.full((T, H * D + 12), 9.0, dtype=torch.bfloat16, device=dev)
    view = fused[:, offset:offset + H * D].unflatten(1, (H, D))
    view.copy_(x.to(dev))
    dp, di, da = pos.to(dev), inv.to(dev), axis.to(dev)
    for inverse in (False, True):
        got = bsa.bsa_rope(view, dp, di, da, interleaved=interleaved, inverse=inverse)
        torch.cuda.synchronize()
        want = oracle.rope(x.double().numpy(), pos.numpy(), inv.numpy(), axis.numpy(), interleaved, inverse)
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= bound(x.double().numpy(), want, 1 << 20, True)).all(), err.max()
        assert torch.equal(got[..., rot:], view[..., rot:])
    bsa.bsa_rope(view, dp, di, da, interleaved=interleaved, inverse=True, out=view)
    torch.cuda.synchronize()
    assert torch.equal(view, got)
    assert (fused[:, :offset] == 9).all() and (fused[:, offset + H * D:] == 9).all()
