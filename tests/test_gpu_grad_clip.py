"""The global gradient norm and clipping against their formulas in 64 bits: mixed types, lengths and
alignments, many tensors, values at the ends of the range, in place and not, graphs, after a backward."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


def _grads(spec, seed=0, scale=1e-2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"b": torch.bfloat16, "f": torch.float32}
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(dt[t]) for t, n in spec]


def _norm64(grads):
    return math.sqrt(sum(g.double().pow(2).sum().item() for g in grads))


def _check_norm(norm, grads):
    want = _norm64(grads)
    # fp32 sums of at most 32 squares (relative error 32 * 2^-24 at most, halved by the root), the result's
    # rounding 2^-24, fp64 elsewhere
    assert abs(norm.item() - want) <= (16 + 1) * 2.0 ** -24 * want * 1.01
    return want


def _check_scaled(outs, grads, max_norm, eps):
    n = _norm64(grads)
    c = min(1.0, max_norm / (n + eps))
    for o, g in zip(outs, grads):
        # the factor is off by the norm's fp32 sums (16 * 2^-24) and its own rounding (2^-24), the product by
        # its fp32 rounding (2^-24) and by the output's
        tol = 19 * 2.0 ** -24 + (torch.finfo(torch.bfloat16).eps / 2 if o.dtype == torch.bfloat16 else 0)
        want = g.double() * c
        assert ((o.double() - want).abs() <= tol * want.abs()).all()


SPECS = {
    "one": [("f", 1)],
    "lengths": [("b", 1), ("f", 3), ("b", 8), ("f", 8192), ("b", 8193), ("f", 8191), ("b", 70001), ("f", 4)],
    "empty-among": [("b", 0), ("f", 1000), ("b", 0), ("b", 77)],
    "many": [("bf"[i % 2], 1 + (i * 37) % 300) for i in range(700)],
    "large": [("b", 30_000_007), ("f", 9_000_001), ("b", 5)],
}


@pytest.mark.parametrize("spec", SPECS)
@pytest.mark.parametrize("max_norm", [0.25, 1e9, float("inf"), 0.0])
def test_clip(moe, spec, max_norm):
    grads = _grads(SPECS[spec])
    keep = [g.clone() for g in grads]
    norm = moe.moe_grad_norm(grads)
    _check_norm(norm, keep)
    out = [torch.full_like(g, 5.0) for g in grads]
    n2, outs = moe.moe_clip_grads(grads, max_norm, out=out)
    assert torch.equal(n2, norm) and all(a is b for a, b in zip(outs, out))
    assert all(torch.equal(g, k) for g, k in zip(grads, keep)), "the inputs were written"
    _check_scaled(out, keep, max_norm, 1e-6)
    n3, same = moe.moe_clip_grads(grads, max_norm)
    assert torch.equal(n3, norm) and all(a is b for a, b in zip(same, grads))
    assert all(torch.equal(g, o) for g, o in zip(grads, out)), "in place differs"


def test_views_off_alignment(moe):
    flat = torch.randn(100_000, device="cuda")
    half = flat.to(torch.bfloat16)
    grads = [flat[1:30_000], flat[30_001:30_004], half[3:9_000], half[9_001:50_000], flat[40_000:90_000]]
    keep = [g.clone() for g in grads]
    rest = flat[90_000:].clone()
    norm, _ = moe.moe_clip_grads(grads, 1.0)
    _check_norm(norm, keep)
    _check_scaled(grads, keep, 1.0, 1e-6)
    assert torch.equal(flat[90_000:], rest)


@pytest.mark.parametrize("value", [1e-20, 1e-30, 1e18, 3e19, 1e38, 1e-40])
def test_range(moe, value):
    """Squares that fp32 cannot hold: the norm of n equal values is value sqrt(n)."""
    n = 40_000
    grads = [torch.full((n,), value, device="cuda"), torch.full((n,), value, device="cuda").to(torch.bfloat16)]
    want = _norm64(grads)
    got = moe.moe_grad_norm(grads).item()
    if want > 3.4028234e38:
        assert got == float("inf")
    else:
        # a result below the normal range is rounded to a multiple of 2^-149
        assert abs(got - want) <= 18 * 2.0 ** -24 * want + 2.0 ** -149


def test_mixed_magnitudes(moe):
    """Small values beside large ones in one thread's group, none lost above the bound."""
    g = torch.full((65536,), 1e-12, device="cuda")
    g[::97] = 3e10
    _check_norm(moe.moe_grad_norm([g]), [g])


@pytest.mark.parametrize("where", [0, 12345, 65535])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_inf(moe, where, dtype):
    g = [torch.ones(65536, device="cuda", dtype=dtype), torch.ones(100, device="cuda")]
    g[0][where] = float("nan")
    norm, out = moe.moe_clip_grads(g, 1.0, out=[torch.zeros_like(t) for t in g])
    assert norm.isnan().all() and all(o.isnan().all() for o in out)
    g[0][where] = -float("inf")
    norm, out = moe.moe_clip_grads(g, 1.0, out=[torch.zeros_like(t) for t in g])
    assert norm.item() == float("inf")
    assert out[0][where].isnan() and int(out[0].isnan().sum()) == 1 and (out[1] == 0).all()


def test_more_than_2_to_31_elements(moe):
    n = 2 ** 31 + 100_003
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[5], g[2 ** 31 - 1], g[2 ** 31 + 1], g[n - 1] = 1.0, 2.0, 4.0, 2.0
    norm, _ = moe.moe_clip_grads([g], 2.5, eps=0.0)
    assert norm.item() == 5.0
    for i, want in ((5, 0.5), (2 ** 31 - 1, 1.0), (2 ** 31 + 1, 2.0), (n - 1, 1.0)):
        assert g[i].item() == want
    assert int((g != 0).sum()) == 4


def test_two_graphs_at_once(moe):
    """Two captured calls replayed on two streams share nothing."""
    sets = [_grads(SPECS["lengths"] + [("f", 2_000_003)], seed=s) for s in (8, 9)]
    graphs, norms = [], [torch.zeros(1, device="cuda") for _ in sets]
    outs = [[torch.empty_like(g) for g in grads] for grads in sets]
    moe.moe_clip_grads(sets[0], 0.5, out=outs[0])
    torch.cuda.synchronize()
    for grads, out, norm in zip(sets, outs, norms):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_clip_grads(grads, 0.5, out=out, norm=norm)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for grads, out, norm in zip(sets, outs, norms):
        _check_norm(norm, grads)
        _check_scaled(out, grads, 0.5, 1e-6)


def test_zero_gradients_and_empty_list(moe):
    g = [torch.zeros(5000, device="cuda"), torch.zeros(0, device="cuda", dtype=torch.bfloat16)]
    norm, out = moe.moe_clip_grads(g, 1.0, eps=0.0)
    assert norm.item() == 0.0 and (out[0] == 0).all()
    norm = torch.full((1,), 3.0, device="cuda")
    assert moe.moe_grad_norm([], norm=norm).item() == 0.0
    norm.fill_(3.0)
    assert moe.moe_clip_grads([], 1.0, norm=norm)[0].item() == 0.0


def test_overlapping_outputs_are_refused(moe):
    buf = torch.ones(1000, device="cuda")
    a, b = buf[:600], buf[500:]
    for args in (([a, b], None), ([a, a], None), ([a.clone(), b.clone()], [a, b]),
                 ([a, b.clone()], [b[:100].clone().resize_(600), a[:500]]), ([buf[1:]], [buf[:-1]])):
        with pytest.raises(moe.MoEError):
            moe.moe_clip_grads(args[0], 1.0, out=args[1])
    assert (buf == 1).all()
    moe.moe_grad_norm([a, b, a])   # reading twice is fine


def test_refusals(moe):
    g, o = [torch.ones(8, device="cuda"), torch.ones(5, device="cuda")], [torch.ones(8, device="cuda")]
    with pytest.raises(ValueError):
        moe.moe_clip_grads(g, 1.0, out=o)                                            # another number
    with pytest.raises(moe.MoEError):
        moe.moe_clip_grads(g, 1.0, out=o + [torch.ones(4, device="cuda")])           # another length
    with pytest.raises(moe.MoEError):
        moe.moe_clip_grads(g, 1.0, out=o + [torch.ones(5, device="cuda").bfloat16()])   # another type
    with pytest.raises(ValueError):
        moe.moe_clip_grads([torch.ones(4, 4, device="cuda").t()], 1.0)               # not contiguous
    with pytest.raises(TypeError):
        moe.moe_clip_grads([torch.ones(4, device="cuda").half()], 1.0)
    with pytest.raises(TypeError):
        moe.moe_clip_grads(g + [torch.ones(4)], 1.0)                                 # on the CPU
    with pytest.raises(TypeError):
        moe.moe_clip_grads(g, 1.0, norm=torch.zeros(1, dtype=torch.float64, device="cuda"))
    for bad in (-1.0, float("nan")):
        with pytest.raises(moe.MoEError):
            moe.moe_clip_grads(g, bad)
    assert all((t == 1).all() for t in g + o)


def test_repeatable_on_another_stream_and_in_a_graph(moe):
    grads = _grads(SPECS["lengths"] + [("b", 3_000_000)], seed=4)
    out = [torch.empty_like(g) for g in grads]
    norm, _ = moe.moe_clip_grads(grads, 0.5, out=out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out2 = [torch.empty_like(g) for g in grads]
        norm2, _ = moe.moe_clip_grads(grads, 0.5, out=out2)
        norm3 = moe.moe_grad_norm(grads)
    norm4, out4 = moe.moe_clip_grads(grads, 0.5, out=[torch.empty_like(g) for g in grads], stream=side)
    side.synchronize()
    assert torch.equal(norm, norm3) and torch.equal(norm, norm4)
    assert all(torch.equal(a, b) for a, b in zip(out, out4))
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(out, out2))
    g = torch.cuda.CUDAGraph()
    nrm = torch.zeros(1, device="cuda")
    with torch.cuda.graph(g):
        moe.moe_clip_grads(grads, 0.5, out=out, norm=nrm)
    for t in grads:
        t.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    _check_norm(nrm, grads)
    _check_scaled(out, grads, 0.5, 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_after_the_layers_backward(moe, dtype):
    """A training step: forward, backward, clip the dict of gradients."""
    import moe_inputs
    from moe_testlib import to_dev, upload
    T, d, F, E, k = 150, 128, 256, 8, 2
    args = upload(moe_inputs.make_inputs(T, d, F, E, k, dtype, seed=41))
    code = moe.MOE_DTYPE_BF16 if dtype == "bf16" else moe.MOE_DTYPE_F32
    ws = torch.empty(moe.moe_train_workspace_size(T, d, F, E, k, code), dtype=torch.uint8, device="cuda")
    moe.moe_forward_ws(*args, k, path=moe.MOE_PATH_TRAIN, workspace=ws)
    g, _ = moe.moe_backward_ws(*args, to_dev(moe_inputs.make_dout(T, d, dtype, seed=41), dtype), k, ws)
    dx = g["dx"].clone()
    keep = [t.clone() for n, t in g.items() if n != "dx"]
    norm, clipped = moe.moe_clip_grads(g, 0.1)
    assert len(clipped) == len(keep) and torch.equal(g["dx"], dx)   # the rows' gradient is no parameter's
    _check_norm(norm, keep)
    _check_scaled(clipped, keep, 0.1, 1e-6)
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_outputs_by_name_and_by_shape(moe):
    """A dict of outputs in another order than the gradients': dW1, dW3 and dW2 have one length and type."""
    g = dict(dx=torch.ones(2, 4, device="cuda"), dWg=torch.full((2, 4), 3.0, device="cuda"),
             dW1=torch.full((2, 6, 4), 1.0, device="cuda"), dW3=torch.full((2, 6, 4), 2.0, device="cuda"),
             dW2=torch.full((2, 4, 6), 4.0, device="cuda"))
    out = {n: torch.zeros_like(g[n]) for n in ("dW2", "dW3", "dW1", "dWg")}
    norm, clipped = moe.moe_clip_grads(g, 1e9, out=out)
    assert all(torch.equal(out[n], g[n]) for n in out)
    assert all(a is out[n] for a, n in zip(clipped, ("dWg", "dW1", "dW3", "dW2")))
    with pytest.raises(ValueError):
        moe.moe_clip_grads([g["dW1"]], 1.0, out=[g["dW2"].clone()])     # one length, another shape
    with pytest.raises(ValueError):
        moe.moe_clip_grads(g, 1.0, out=dict(out, dW2=torch.zeros(2, 6, 4, device="cuda")))
    with pytest.raises(TypeError):
        moe.moe_clip_grads([g["dW1"]], 1.0, out=[torch.zeros(2, 6, 4)])                                # on the CPU
    with pytest.raises(moe.MoEError):
        moe.moe_clip_grads([g["dW1"]], 1.0, out=[torch.zeros(2, 6, 4, device="cuda").bfloat16()])      # another type


@pytest.mark.parametrize("value,max_norm", [(1e38, 1e-3), (1e38, 1e-6), (3e38, 1.0), (2e30, 1e-12), (1e38, 1e-30),
                                            (1e-20, 1e-30)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_factors_below_the_normal_range(moe, value, max_norm, dtype):
    """c = max_norm / n may be below fp32's normal range while c g is in it; n may be above fp32's range.  Values
    of all lengths: vectors, their rests, and off 16-byte alignment."""
    buf = torch.full((9001,), value, device="cuda").to(dtype)
    grads = [buf[:5003].clone(), buf[1:4000], torch.tensor([value / 3, -value], device="cuda")]
    keep = [g.clone() for g in grads]
    norm, outs = moe.moe_clip_grads(grads, max_norm, eps=0.0, out=[torch.empty_like(g) for g in grads])
    n = _norm64(keep)
    if n > 3.4028234e38:
        assert norm.item() == float("inf")
    c = min(1.0, torch.tensor(max_norm).double().item() / n)   # (max_norm travels as a float)
    for o, g in zip(outs, keep):
        # as _check_scaled; a result below the normal range is rounded to a multiple of the type's smallest, twice
        # (the product, then the output)
        tiny = 2.0 ** -149 if o.dtype == torch.float32 else 2.0 ** -133
        tol = 19 * 2.0 ** -24 + (torch.finfo(torch.bfloat16).eps / 2 if o.dtype == torch.bfloat16 else 0)
        want = g.double() * c
        assert ((o.double() - want).abs() <= tol * want.abs() + tiny).all()


def test_infinite_max_norm_leaves_infinite_gradients(moe):
    g = [torch.tensor([1.0, float("inf"), -3.0], device="cuda"), torch.ones(40, device="cuda").bfloat16()]
    norm, outs = moe.moe_clip_grads(g, float("inf"), out=[torch.zeros_like(t) for t in g])
    assert norm.item() == float("inf") and all(torch.equal(o, t) for o, t in zip(outs, g))
    g[1][7] = float("nan")
    norm, outs = moe.moe_clip_grads(g, float("inf"), out=outs)
    assert norm.isnan().all() and all(o.isnan().all() for o in outs)


def test_a_factor_just_below_a_power_of_two(moe):
    """c = 2^-110 (1 - 2^-40) rounds to a power of two in fp32: in place it still scales."""
    g = [torch.zeros(64, device="cuda")]
    g[0][3] = 2.0 ** 100 * (1 + 2.0 ** -20)
    want = g[0].double() * (2.0 ** -10 / (2.0 ** 100 * (1 + 2.0 ** -20)))
    norm, _ = moe.moe_clip_grads(g, 2.0 ** -10, eps=0.0)
    assert ((g[0].double() - want).abs() <= 19 * 2.0 ** -24 * want.abs()).all()
    g = [torch.zeros(64, device="cuda")]
    g[0][3] = 2.0 ** 100
    moe.moe_clip_grads(g, 2.0 ** -10 * (1 - 2.0 ** -24), eps=0.0)
    assert abs(g[0][3].item() - 2.0 ** -10) <= 19 * 2.0 ** -34
