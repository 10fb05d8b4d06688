"""Second derivatives through the grouped product's autograd functions are right, those of the layer raise; neither
are dropped.  The kernels are replaced by torch products: no GPU needed."""
import pytest
import torch

import sparse_mixture_experts_14_b200.nn as nn


@pytest.fixture
def products(monkeypatch):
    def segs(off):
        off = off.tolist()
        return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(off, off[1:]))]

    # (as the kernels: nothing they do is recorded)
    @torch.no_grad()
    def mm(x, W, off, counts=None, out=None):
        for e, r in segs(off):
            out[r] = x[r] @ W[e].t()
        return out

    @torch.no_grad()
    def dgrad(dy, W, off, counts=None, out=None):
        for e, r in segs(off):
            out[r] = dy[r] @ W[e]
        return out

    @torch.no_grad()
    def wgrad(dy, x, off, counts=None):
        return torch.stack([dy[r].t() @ x[r] for _, r in segs(off)])

    monkeypatch.setattr(nn, "moe_grouped_mm", mm)
    monkeypatch.setattr(nn, "moe_grouped_dgrad", dgrad)
    monkeypatch.setattr(nn, "moe_grouped_wgrad", wgrad)


@pytest.mark.parametrize("second", ["square", "linear"])
def test_grouped_linear(products, second):
    """A gradient penalty: its derivative by W and x, against the same in torch's own products."""
    torch.manual_seed(1)
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    lin = nn.GroupedLinear(2, 4, 6, dtype=torch.float32, device="cpu")
    x = torch.randn(5, 4, requires_grad=True)

    def loss(y, x, W):
        first = y.pow(2).sum() if second == "square" else y.sum()
        dx, dW = torch.autograd.grad(first, (x, W), create_graph=True)
        return y.sum() + dx.pow(2).sum() + (dW * dW.detach().cos()).sum()

    got = torch.autograd.grad(loss(lin(x, off), x, lin.W), (x, lin.W))
    plain = torch.cat([x[:3] @ lin.W[0].t(), x[3:] @ lin.W[1].t()])
    want = torch.autograd.grad(loss(plain, x, lin.W), (x, lin.W))
    for g, w in zip(got, want):
        assert torch.allclose(g, w, rtol=1e-4, atol=1e-5)




def test_layer(monkeypatch):
    def forward(x, *weights, path, workspace):
        return x * 2

    def backward(x, Wg, W1, W3, W2, dout, k, ws, alpha, wgrad_dtype):
        return dict(dx=dout * 2, dWg=torch.zeros_like(Wg), dW1=torch.zeros_like(W1), dW3=torch.zeros_like(W3),
                    dW2=torch.zeros_like(W2)), 0

    monkeypatch.setattr(nn, "moe_forward_ws", forward)
    monkeypatch.setattr(nn, "moe_backward_ws", backward)
    layer = nn.SparseMoE(8, 16, E=4, k=2, dtype=torch.float32, device="cpu")
    x = torch.randn(3, 8, requires_grad=True)
    dx, = torch.autograd.grad(layer(x).sum(), x, create_graph=True)
    assert torch.equal(dx, torch.full_like(x, 2))
    with pytest.raises(RuntimeError, match="second derivatives"):
        (dx.pow(2).sum() + x.sum()).backward()
    # the first derivatives with a graph that nobody follows
    out = layer(x)
    out.sum().backward(create_graph=True)
    assert torch.equal(x.grad.detach(), torch.full_like(x, 2)) and layer.W1.grad is not None
