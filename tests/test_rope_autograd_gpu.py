"""rope under autograd."""
import numpy as np
import pytest
import torch

from tests.cache_fp8_common import DEV, bf16, ints

pytestmark = pytest.mark.gpu


def _inputs(fa, B=2, H=3, N=37, d=64, rot=32, seed=0):
    rng = np.random.default_rng(seed)
    x, g = bf16(rng, (B, H, N, d)).to(DEV), bf16(rng, (B, H, N, d)).to(DEV)
    return x, g, fa.rope_table(10000.0 ** (-2.0 * np.arange(rot // 2) / rot)), ints(rng.integers(0, 5000, (B, N)))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_records_its_gradient(cuda_lib, inter, inverse):
    x, g, table, pos = _inputs(cuda_lib)
    plain = cuda_lib.rope(x, table, pos, inter, 1.25, inverse)
    x.requires_grad_()
    y = cuda_lib.rope(x, table, pos, inter, 1.25, inverse)
    assert y.requires_grad and torch.equal(y, plain)
    want = cuda_lib.rope(g, table, pos, inter, 1.25, not inverse)
    got, = torch.autograd.grad(y, x, g)
    assert torch.equal(got, want)
    # the map is linear: the gradient of <dx, u> by g is the rotation of u
    g2 = g.clone().requires_grad_()
    y = cuda_lib.rope(x, table, pos, inter, 1.25, inverse)
    dx, = torch.autograd.grad(y, x, g2, create_graph=True)
    u = torch.flip(g, (2,))
    back, = torch.autograd.grad(dx, g2, u)
    assert torch.equal(back, cuda_lib.rope(u, table, pos, inter, 1.25, inverse))
    with torch.no_grad():
        assert not cuda_lib.rope(x, table, pos, inter, 1.25, inverse).requires_grad


def test_rope_gradients_of_any_layout(cuda_lib):
    """Gradients that arrive expanded, token-major, in rows that the kernel does not take, or at an odd address; heads
    that share an input; a side stream."""
    x, g, table, pos = _inputs(cuda_lib, N=40)
    x.requires_grad_()
    want = cuda_lib.rope(g, table, pos, inverse=True)
    odd = torch.empty(g.numel() + 1, dtype=g.dtype, device=DEV)[1:].view(g.shape).copy_(g)
    rows = torch.empty(g.shape[:3] + (68,), dtype=g.dtype, device=DEV)[..., :64].copy_(g)
    for grad in (g, g.transpose(1, 2).contiguous().transpose(1, 2), g.transpose(2, 3).contiguous().transpose(2, 3), odd, rows):
        got, = torch.autograd.grad(cuda_lib.rope(x, table, pos), x, grad)
        assert torch.equal(got, want)
    ones = torch.ones_like(g)
    cuda_lib.rope(x, table, pos).sum().backward()
    assert torch.equal(x.grad, cuda_lib.rope(ones, table, pos, inverse=True))
    one = x.detach()[:, :1].clone().requires_grad_()
    got, = torch.autograd.grad(cuda_lib.rope(one.expand(-1, 3, -1, -1), table, pos), one, g)
    assert torch.equal(got, want.sum(1, keepdim=True))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = cuda_lib.rope(x, table, pos, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    got, = torch.autograd.grad(y, x, g)
    assert torch.equal(got, want)


def test_rope_gradient_captured(cuda_lib):
    x, g, table, pos = _inputs(cuda_lib)
    x.requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(cuda_lib.rope(x, table, pos), x, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cuda_lib.rope(x, table, pos)
        dx, = torch.autograd.grad(y, x, g)
    g.copy_(torch.flip(g, (1,)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, cuda_lib.rope(x.detach(), table, pos)) and torch.equal(dx, cuda_lib.rope(g, table, pos, inverse=True))


def test_rope_refuses_out_where_a_gradient_is_recorded(cuda_lib):
    x, g, table, pos = _inputs(cuda_lib)
    x.requires_grad_()
    out = torch.empty_like(g)
    for a, b in ((x, out), (g, out.clone().requires_grad_()), (x, x)):
        with pytest.raises(ValueError):
            cuda_lib.rope(a, table, pos, out=b)
    with torch.no_grad():
        cuda_lib.rope(x, table, pos, out=out)
    assert torch.equal(out, cuda_lib.rope(x.detach(), table, pos))
