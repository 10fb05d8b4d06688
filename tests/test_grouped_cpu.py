"""The grouped products, the adapters and the gradient clipping without a GPU: argument checks of the C ABI
(nothing is launched) and of the binding."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    return ctypes.CDLL(__graft_entry__._builder().build())


def _p(v):
    return ctypes.c_void_p(v)


def _mm(lib, name="moe_grouped_mm", a=0x1000, b=0x2000, off=0x3000, cnt=0, out=0x4000, M=10, N=64, K=64, E=4, dt=1,
        odt=1):
    return getattr(lib, name)(_p(a), _p(b), _p(off), _p(cnt), _p(out), M, N, K, E, dt, odt, None)


@pytest.mark.parametrize("name", ["moe_grouped_mm", "moe_grouped_dgrad", "moe_grouped_wgrad"])
def test_grouped_argument_checks(lib, name):
    f = lambda **kw: _mm(lib, name, **kw)
    assert f(M=-1) == INVALID
    assert f(N=0) == INVALID and f(K=-8) == INVALID and f(E=0) == INVALID
    assert f(dt=2) == INVALID and f(dt=-1) == INVALID
    assert f(dt=0, odt=1) == INVALID            # float inputs give float
    assert f(odt=7) == INVALID
    assert f(E=257) == UNSUPPORTED
    assert f(N=60) == UNSUPPORTED and f(K=4) == UNSUPPORTED
    assert f(dt=0, odt=0, N=62) == UNSUPPORTED
    assert f(off=0) == INVALID and f(off=0x3002) == INVALID and f(cnt=0x3001) == INVALID
    assert f(a=0) == INVALID and f(b=0) == INVALID and f(out=0) == INVALID
    assert f(a=0x1008) == INVALID and f(b=0x2004) == INVALID and f(out=0x4002) == INVALID
    assert f(M=2 ** 31 - 1) == UNSUPPORTED
    if name != "moe_grouped_wgrad":
        assert f(M=0, a=0, out=0) == 0          # no rows: a no-op


def _lora(lib, x=0x1000, off=0x3000, A=0x5000, B=0x6000, scale=0x7000, ids=0x8000, M=10, N=64, K=64, E=4, L=3, R=16,
          odt=1, ws=0x10000, wsb=1 << 30):
    return lib.moe_grouped_lora(_p(x), _p(0x2000), _p(off), _p(0), _p(A), _p(B), _p(scale), _p(ids), _p(0x4000), M, N,
                                K, E, L, R, odt, _p(ws), ctypes.c_size_t(wsb), None)


def test_lora_argument_checks(lib):
    lib.moe_grouped_lora_workspace_size.restype = ctypes.c_size_t
    size = lib.moe_grouped_lora_workspace_size
    assert size(10, 4, 3, 16) >= 10 * 16 * 2 and size(1000, 4, 3, 16) > size(10, 4, 3, 16)
    assert size(-1, 4, 3, 16) == 0 and size(10, 0, 3, 16) == 0 and size(10, 4, 0, 16) == 0
    assert size(10, 4, 3, 12) == 0 and size(10, 4, 3, 136) == 0 and size(10, 257, 3, 16) == 0
    f = lambda **kw: _lora(lib, **kw)
    assert f(R=12) == UNSUPPORTED and f(R=136) == UNSUPPORTED and f(R=0) == INVALID
    assert f(L=0) == INVALID and f(L=2 ** 30) == UNSUPPORTED
    assert f(A=0) == INVALID and f(B=0) == INVALID and f(scale=0) == INVALID and f(ids=0) == INVALID
    assert f(A=0x5008) == INVALID and f(B=0x6008) == INVALID and f(ids=0x8002) == INVALID
    assert f(ws=0) == WORKSPACE and f(ws=0x10010) == WORKSPACE and f(wsb=16) == WORKSPACE
    assert f(M=-1) == INVALID and f(odt=3) == INVALID and f(N=12) == UNSUPPORTED and f(off=0) == INVALID
    assert f(M=0, A=0) == 0


class Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


def _list(*t):
    arr = (Tensor * max(len(t), 1))()
    for d, (p, n, k) in zip(arr, t):
        d.data, d.numel, d.dtype = p, n, k
    return arr


def _clip(lib, g, out=None, n=None, max_norm=1.0, eps=1e-6, norm=0x9000):
    return lib.moe_clip_grads(g, out, len(g) if n is None else n, ctypes.c_float(max_norm), ctypes.c_float(eps),
                              _p(norm), None)


def test_clip_argument_checks(lib):
    g = _list((0x1000, 100, 0), (0x2000, 50, 1))
    assert _clip(lib, g, n=-1) == INVALID and _clip(lib, None, n=2) == INVALID
    assert _clip(lib, g, norm=0) == INVALID and _clip(lib, g, norm=0x9002) == INVALID
    assert _clip(lib, g, max_norm=-1.0) == INVALID and _clip(lib, g, max_norm=float("nan")) == INVALID
    assert _clip(lib, g, eps=-1.0) == INVALID and _clip(lib, g, eps=float("inf")) == INVALID
    for bad in ((0x1000, -1, 0), (0x1000, 4, 2), (0, 4, 0), (0x1002, 4, 0), (0x1001, 4, 1)):
        assert _clip(lib, _list(bad)) == INVALID
        assert lib.moe_grad_norm(_list(bad), 1, _p(0x9000), None) == INVALID
    assert _clip(lib, g, _list((0x5000, 100, 0), (0x6000, 49, 1))) == INVALID     # another length
    assert _clip(lib, g, _list((0x5000, 100, 0), (0x6000, 50, 0))) == INVALID     # another type
    # overlaps: the same tensor twice, outputs over one another, over another input, shifted over its own
    assert _clip(lib, _list((0x1000, 100, 0), (0x1000, 100, 0))) == INVALID
    assert _clip(lib, _list((0x1000, 100, 0), (0x1100, 100, 0))) == INVALID
    assert _clip(lib, g, _list((0x5000, 100, 0), (0x5180, 50, 1))) == INVALID
    assert _clip(lib, g, _list((0x2000, 100, 0), (0x6000, 50, 1))) == INVALID
    assert _clip(lib, g, _list((0x1010, 100, 0), (0x6000, 50, 1))) == INVALID
    assert lib.moe_grad_norm(g, 2, _p(0), None) == INVALID


def test_binding_checks():
    import sparse_mixture_experts_14_b200 as moe
    x, W = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 32, 64, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        moe.moe_grouped_mm(x, W, off)                       # CPU tensors
    with pytest.raises(ValueError):
        moe.moe_grouped_mm(x, W, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.moe_grouped_mm(x, W, off, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.moe_clip_grads([], 1.0)
    with pytest.raises(TypeError):
        moe.moe_clip_grads([x], 1.0)
    with pytest.raises(TypeError):
        moe.moe_clip_grads([x], 1.0, out=[x[:2]])
    with pytest.raises(TypeError):
        moe.moe_clip_grads([3.0], 1.0)
