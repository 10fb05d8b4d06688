"""Second derivatives through the layer's and the grouped product's autograd functions raise; they are not
dropped.  The kernels are replaced by torch products: no GPU needed."""
import pytest
import torch

import sparse_mixture_experts_14_b200.nn as nn


@pytest.fixture
def products(monkeypatch):
    def segs(off):
        off = off.tolist()
        return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(off, off[1:]))]

    def mm(x, W, off, counts=None, out=None):
        for e, r in segs(off):
            out[r] = x[r] @ W[e].t()
        return out

    def dgrad(dy, W, off, counts=None, out=None):
        for e, r in segs(off):
            out[r] = dy[r] @ W[e]
        return out

    def wgrad(dy, x, off, counts=None):
        return torch.stack([dy[r].t() @ x[r] for _, r in segs(off)])

    monkeypatch.setattr(nn, "moe_grouped_mm", mm)
    monkeypatch.setattr(nn, "moe_grouped_dgrad", dgrad)
    monkeypatch.setattr(nn, "moe_grouped_wgrad", wgrad)


def test_grouped_linear(products):
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    lin = nn.GroupedLinear(2, 4, 6, dtype=torch.float32, device="cpu")
    x = torch.randn(5, 4, requires_grad=True)
    y = lin(x, off)
    dx, = torch.autograd.grad(y.sum(), x, create_graph=True)
    want = torch.cat([lin.W[0].sum(0).expand(3, 4), lin.W[1].sum(0).expand(2, 4)])
    assert torch.allclose(dx, want)                      # a first derivative as ever
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx.pow(2).sum() + lin(x, off).sum()).backward()


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
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (dx.pow(2).sum() + x.sum()).backward()
