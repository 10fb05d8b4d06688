"""GroupedLinear and clip_grad_norm_: autograd over the grouped products, with the layer's dispatch, and a
training step captured into a graph while an eager graph of the same parameters lives."""
import pytest
import torch

from grouped_testlib import DT, check, mm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    import sparse_mixture_experts_14_b200 as m
    import sparse_mixture_experts_14_b200.nn as nn
    return m, nn


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients(mods, dtype):
    moe, nn = mods
    counts = [70, 0, 3]
    off = torch.tensor([0, 128, 128, 140], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    torch.manual_seed(3)
    lin = nn.GroupedLinear(3, 72, 40, dtype=DT[dtype])
    x = torch.randn(140, 72, device="cuda").to(DT[dtype]).requires_grad_()
    dy = torch.randn(140, 40, device="cuda").to(DT[dtype])
    y = lin(x, off, cnt)
    y.backward(dy)
    gap = [r for r in range(140) if not (r < 70 or 128 <= r < 131)]
    assert (y[gap] == 0).all() and (x.grad[gap] == 0).all()
    for e, (s, n) in enumerate(zip([0, 128, 128], counts)):
        r = slice(s, s + n)
        W = lin.W.detach()[e]
        check(y.detach()[r], *mm(x.detach()[r], W.t()), 72, "y")
        check(x.grad[r], *mm(dy[r], W), 40, "dx")
        check(lin.W.grad[e], *mm(dy[r].t(), x.detach()[r]), n, "dW")
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_only_the_asked_gradients(mods):
    moe, nn = mods
    off = torch.tensor([0, 5, 9], dtype=torch.int32, device="cuda")
    lin = nn.GroupedLinear(2, 64, 64)
    x = torch.randn(9, 64, device="cuda", dtype=torch.bfloat16)
    lin(x, off).float().sum().backward()
    assert lin.W.grad is not None
    lin.W.requires_grad_(False)
    lin.W.grad = None
    x.requires_grad_()
    lin(x, off).float().sum().backward()
    assert x.grad is not None and lin.W.grad is None


def test_training_step_in_a_graph(mods):
    """Two grouped layers, their gradients and the clip, captured; an eager step before gives the same."""
    moe, nn = mods
    torch.manual_seed(5)
    off = torch.tensor([0, 40, 47, 47, 200], dtype=torch.int32, device="cuda")
    a, b = nn.GroupedLinear(4, 128, 256), nn.GroupedLinear(4, 256, 128)
    params = [a.W, b.W]
    x = torch.randn(200, 128, device="cuda", dtype=torch.bfloat16)

    def step():
        y = b(torch.relu(a(x, off)), off)
        grads = torch.autograd.grad(y.float().pow(2).sum(), params)
        return moe.moe_clip_grads(list(grads), 1.0)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            norm, eager = step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gnorm, captured = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, gnorm) and all(torch.equal(p, q) for p, q in zip(eager, captured))
    total = sum(t.double().pow(2).sum().item() for t in captured) ** 0.5
    assert abs(total - 1.0) <= 2.0 ** -8   # every clipped gradient rounded to bf16
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_clip_grad_norm_on_the_layer(mods):
    moe, nn = mods
    torch.manual_seed(6)
    layer = nn.SparseMoE(d=128, ffn=256, E=8, k=2)
    layer(torch.randn(64, 128, device="cuda", dtype=torch.bfloat16)).float().pow(2).sum().backward()
    keep = [p.grad.clone() for p in layer.parameters()]
    want = sum(t.double().pow(2).sum().item() for t in keep) ** 0.5
    norm = nn.clip_grad_norm_(layer.parameters(), want / 4)
    assert abs(norm.item() - want) <= 18 * 2.0 ** -24 * want
    for p, k in zip(layer.parameters(), keep):
        w = k.double() * (want / 4 / (want + 1e-6))
        assert ((p.grad.double() - w).abs() <= (2.0 ** -8 + 2.0 ** -18) * w.abs()).all()
    assert nn.clip_grad_norm_([torch.nn.Parameter(torch.ones(3, device="cuda"))], 1.0).item() == 0.0


def test_second_derivatives(mods):
    """sum (dL/dx)^2 of L = sum y^2 / 2, by W and by x, in fp32 against the formula in 64 bits: with
    G_e = W_e^T W_e, dL/dx_r = G_e x_r, so the penalty is sum |G x|^2."""
    moe, nn = mods
    counts, starts = [33, 0, 70], [0, 33, 40]
    off = torch.tensor(starts + [110], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    torch.manual_seed(7)
    lin = nn.GroupedLinear(3, 72, 40, dtype=torch.float32)
    x = torch.randn(110, 72, device="cuda", requires_grad=True)
    y = lin(x, off, cnt)
    dx, = torch.autograd.grad(y.pow(2).sum() / 2, x, create_graph=True)
    gx, gW = torch.autograd.grad(dx.pow(2).sum(), (x, lin.W))
    W64 = lin.W.detach().double().requires_grad_()
    x64 = x.detach().double().requires_grad_()
    live = torch.zeros(110, dtype=torch.bool, device="cuda")
    pen = 0.0
    for e, (s, n) in enumerate(zip(starts, counts)):
        live[s:s + n] = True
        pen = pen + (x64[s:s + n] @ W64[e].t() @ W64[e]).pow(2).sum()
    wx, wW = torch.autograd.grad(pen, (x64, W64))
    assert (gx[~live] == 0).all() and (gW[1] == 0).all()
    # chains of at most five products of up to 110 terms each, every one within (n + 8) 2^-23 of its magnitudes; the
    # magnitudes of a random chain exceed its values by sqrt(n) < 11 a product at most
    for g, w in ((gx, wx), (gW, wW)):
        assert (g.double() - w).abs().max() <= 5 * 118 * 2.0 ** -23 * 11 * w.abs().max()
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_clip_grad_norm_without_gradients(mods):
    moe, nn = mods
    p = torch.nn.Parameter(torch.ones(3, device="cuda"))
    norm = nn.clip_grad_norm_([p], 1.0)
    assert norm.device == p.device and norm.dtype == torch.float32 and norm.item() == 0.0
    assert nn.clip_grad_norm_(iter([]), 1.0).item() == 0.0


def test_clip_grad_norm_of_gradients_of_any_strides(mods):
    """Transposed and permuted gradients, one with gaps between its rows, one of stride 2: as torch's clip."""
    moe, nn = mods
    torch.manual_seed(8)
    grads = [torch.randn(6, 10, device="cuda").t(), torch.randn(3, 4, 5, device="cuda").permute(2, 0, 1),
             torch.randn(7, 16, device="cuda")[:, :9], torch.randn(22, device="cuda").bfloat16()[::2],
             torch.randn(5, device="cuda"), torch.randn(1, 4, device="cuda").expand(1, 4), torch.randn((), device="cuda")]
    gaps = grads[2]._base[:, 9:].clone()
    params = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
    for p, g in zip(params, grads):
        p.grad = g
    keep = [g.clone() for g in grads]
    want = sum(k.double().pow(2).sum().item() for k in keep) ** 0.5
    norm = nn.clip_grad_norm_(params, want / 3)
    assert abs(norm.item() - want) <= 18 * 2.0 ** -24 * want
    for p, g, k in zip(params, grads, keep):
        assert p.grad is g
        w = k.double() * (want / 3 / (want + 1e-6))
        tol = 19 * 2.0 ** -24 + (2.0 ** -8 if g.dtype == torch.bfloat16 else 0)
        assert ((g.double() - w).abs() <= tol * w.abs()).all()
    assert torch.equal(grads[2]._base[:, 9:], gaps)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_off_alignment(mods, dtype):
    """The output goes into a concatenation behind one value: its gradient is contiguous at an odd offset; so is x."""
    moe, nn = mods
    torch.manual_seed(9)
    off = torch.tensor([0, 20, 31], dtype=torch.int32, device="cuda")
    lin = nn.GroupedLinear(2, 64, 40, dtype=DT[dtype])
    x = torch.randn(1 + 31 * 64, device="cuda").to(DT[dtype])[1:].view(31, 64).requires_grad_()
    dz = torch.randn(1 + 31 * 40, device="cuda").to(DT[dtype])
    y = lin(x, off)
    torch.cat([torch.zeros(1, device="cuda", dtype=DT[dtype]), y.flatten()]).backward(dz)
    dy = dz[1:].view(31, 40)
    for e, r in enumerate((slice(0, 20), slice(20, 31))):
        W = lin.W.detach()[e]
        check(y.detach()[r], *mm(x.detach()[r], W.t()), 64, "y")
        check(x.grad[r], *mm(dy[r], W), 40, "dx")
        check(lin.W.grad[e], *mm(dy[r].t(), x.detach()[r]), dy[r].shape[0], "dW")
    layer = nn.SparseMoE(d=128, ffn=256, E=8, k=2)
    h = torch.randn(1 + 16 * 128, device="cuda").bfloat16()
    a = layer(h[1:].view(16, 128))
    assert torch.equal(a, layer(h[1:].view(16, 128).clone()))
    torch.cat([h[:1], a.flatten()]).sum().backward()
    assert torch.isfinite(layer.W1.grad).all()
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_empty_batch(mods):
    moe, nn = mods
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    lin = nn.GroupedLinear(3, 64, 40)
    x = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = lin(x, off)
    y.sum().backward()
    assert y.shape == (0, 40) and x.grad.shape == (0, 64) and (lin.W.grad == 0).all()
