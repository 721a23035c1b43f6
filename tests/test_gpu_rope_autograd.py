"""bsa_rope within autograd.  Gradients are those of the transposed map, within the
tolerance of tests/test_gpu_rope.py."""
import numpy as np
import pytest
import torch

import block_sparse_attention_topk_gb300 as bsa
import oracle
from tests.test_gpu_rope import _case, bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_reaches_the_leaf(cuda_device, dtype, interleaved, inverse):
    T, H, D, rot = 19, 3, 64, 48
    x, pos, inv, axis = _case(T, H, D, rot, 2, dtype, 3)
    w = torch.randn((T, H, D), generator=torch.Generator().manual_seed(4)).to(dtype)
    dev = cuda_device
    leaf = x.to(dev).requires_grad_()
    args = (pos.to(dev), inv.to(dev), axis.to(dev), interleaved, inverse)
    y = bsa.bsa_rope(leaf, *args)
    assert y.requires_grad and torch.equal(y.detach(), bsa.bsa_rope(x.to(dev), *args))
    (y * w.to(dev)).sum().backward()
    want = oracle.rope(w.double().numpy(), pos.numpy(), inv.numpy(), axis.numpy(), interleaved, not inverse)
    err = np.abs(leaf.grad.double().cpu().numpy() - want)
    assert (err <= bound(w.double().numpy(), want, 1 << 20, dtype == torch.bfloat16)).all()


def test_gradient_of_strided_and_broadcast_inputs(cuda_device):
    """Parts of a fused buffer; one head broadcast to several; an output whose
    gradient is an expanded scalar; against differences (the map is linear)."""
    T, H, D = 7, 4, 32
    x, pos, inv, _ = _case(T, 3 * H, D, D, 1, torch.float32, 5)
    dev = cuda_device
    pd, fd = pos[0].to(dev), inv.to(dev)
    fused = x.to(dev).requires_grad_()
    bsa.bsa_rope(fused[:, H:2 * H], pd, fd).sum().backward()
    one = np.ones((T, H, D))
    want = oracle.rope(one, pos.numpy(), inv.numpy(), inverse=True)
    got = fused.grad.double().cpu().numpy()
    assert (np.abs(got[:, H:2 * H] - want) <= bound(one, want, 1 << 20, False)).all()
    assert (got[:, :H] == 0).all() and (got[:, 2 * H:] == 0).all()
    head = x[:, :1].to(dev).requires_grad_()
    w = torch.randn((T, H, D), generator=torch.Generator().manual_seed(6))
    (bsa.bsa_rope(head.expand(T, H, D), pd, fd) * w.to(dev)).sum().backward()
    want = oracle.rope(w.double().numpy(), pos.numpy(), inv.numpy(), inverse=True)
    tol = bound(w.double().numpy(), want, 1 << 20, False).sum(1) + 3 * 2.0 ** -24 * np.abs(want).sum(1)
    assert (np.abs(head.grad.double().cpu().numpy()[:, 0] - want.sum(1)) <= tol).all()
    step = np.random.default_rng(7).standard_normal((T, 1, D))
    base = np.broadcast_to(x[:, :1].double().numpy(), (T, H, D))
    diff = (oracle.rope(base + step, pos.numpy(), inv.numpy()) - oracle.rope(base - step, pos.numpy(), inv.numpy())) / 2
    moved = (head.grad.double().cpu().numpy() * step).sum()
    assert abs(moved - (diff * w.double().numpy()).sum()) <= T * D * tol.max() * np.abs(step).max() + 1e-9


def test_second_derivatives(cuda_device):
    T, H, D = 3, 2, 16
    x, pos, inv, _ = _case(T, H, D, D, 1, torch.float32, 8)
    leaf = x.to(cuda_device).requires_grad_()
    y = bsa.bsa_rope(leaf, pos[0].to(cuda_device), inv.to(cuda_device))
    g, = torch.autograd.grad((y ** 3).sum(), leaf, create_graph=True)
    assert g.requires_grad
    gg, = torch.autograd.grad((g * g).sum(), leaf)
    # d/dx sum (R^T 3 y^2)^2 = R^T (36 y^3) for a rotation R
    want = bsa.bsa_rope(36 * y.detach() ** 3, pos[0].to(cuda_device), inv.to(cuda_device), inverse=True)
    assert torch.allclose(gg, want, rtol=1e-4, atol=1e-3)


def test_what_has_no_gradient_is_refused(cuda_device):
    dev = cuda_device
    x, pos, inv, _ = _case(4, 2, 16, 16, 1, torch.float32, 9)
    pd, fd = pos[0].to(dev), inv.to(dev)
    leaf = x.to(dev).requires_grad_()
    for kw in (dict(out=torch.empty_like(leaf)), dict(out=leaf)):
        with pytest.raises(ValueError, match="out"):
            bsa.bsa_rope(leaf, pd, fd, **kw)
    with pytest.raises(ValueError, match="inv_freq"):
        bsa.bsa_rope(x.to(dev), pd, fd.clone().requires_grad_())
    with torch.no_grad():
        place = leaf.clone()
        assert bsa.bsa_rope(place, pd, fd, out=place) is place
        assert not bsa.bsa_rope(leaf, pd, fd).requires_grad


def test_writing_calls_count_as_changes(cuda_device):
    """A tensor that a graph has saved and a call then writes to is found out."""
    dev = cuda_device
    x, pos, inv, _ = _case(4, 2, 16, 16, 1, torch.float32, 10)
    pd, fd = pos[0].to(dev), inv.to(dev)
    buf = x.to(dev)
    w = torch.ones_like(buf, requires_grad=True)
    y = (w * buf).sum()
    before = buf._version
    bsa.bsa_rope(buf, pd, fd, out=buf)
    assert buf._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    kv = torch.randn((2, 1, 16), device=dev).to(torch.bfloat16)
    caches = [torch.zeros((8, 16, 1, 16), dtype=torch.float8_e4m3fn, device=dev) for _ in range(2)]
    scales = [torch.ones((8, 1), device=dev) for _ in range(2)]
    q_out = torch.empty_like(kv)
    old = [t._version for t in (*caches, *scales, q_out)]
    bsa.bsa_append_kv_decode(kv, kv, *caches, torch.zeros((1, 1), dtype=torch.int32, device=dev),
                             torch.tensor([2], dtype=torch.int32, device=dev), 2, q=kv, k_scale=scales[0],
                             v_scale=scales[1], q_out=q_out)
    assert all(t._version > v for t, v in zip((*caches, *scales, q_out), old))
    with torch.inference_mode():
        frozen = x.to(dev)
    bsa.bsa_rope(frozen, pd, fd, out=frozen)       # no counter to move
    torch.cuda.synchronize()


def test_gradient_in_a_graph(cuda_device):
    """Forward and backward captured together, replayed on new inputs."""
    T, H, D = 33, 2, 64
    x, pos, inv, _ = _case(T, H, D, D, 1, torch.bfloat16, 11)
    dev = cuda_device
    pd, fd = pos[0].to(dev), inv.to(dev)
    leaf = x.to(dev).requires_grad_()
    w = torch.ones_like(leaf, requires_grad=False)
    stream = torch.cuda.Stream(dev)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.autograd.grad((bsa.bsa_rope(leaf, pd, fd) * w).sum(), leaf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        g, = torch.autograd.grad((bsa.bsa_rope(leaf, pd, fd) * w).sum(), leaf)
    for seed in range(2):
        w.copy_(torch.randn(w.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(g, bsa.bsa_rope(w, pd, fd, inverse=True))
