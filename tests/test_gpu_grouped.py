"""The ragged grouped products against their formulas in 64 bits: segments of every kind (empty, one
row, across tile borders, gaps), odd sizes, both types, every direction; NaN and Inf stay in their own
rows; rows of no segment keep what they held; streams, graphs, the layer's own dispatch."""
import pytest
import torch

from grouped_testlib import DT, check, device_segments, mm, randn, segments

pytestmark = pytest.mark.gpu

SENTINEL = -77.0


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


# (rows of each expert, alignment of the segments, rows before and after, counts given)
SEGMENTS = {
    "one-row": ([1], 1, 0, 0, False),
    "empty-all": ([0, 0, 0], 1, 0, 5, True),
    "mixed": ([0, 5, 0, 130, 1, 0], 1, 0, 0, False),
    "tiles": ([256, 1, 257, 31, 33, 128], 1, 3, 9, True),
    "padded": ([40, 0, 129, 64], 128, 0, 128, True),
    "long": ([700, 3], 1, 0, 0, False),
    "many": ([(7 * e) % 5 for e in range(64)], 1, 1, 2, False),
    "few-rows": ([3, 0, 2, 1, 4, 0, 1, 2], 1, 0, 0, False),
    "max-experts": ([1 if e % 3 == 0 else 0 for e in range(256)], 1, 0, 0, True),
}
SIZES = [(264, 72), (8, 520), (776, 8), (128, 256), (40, 1032)]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


def _inputs(seg, N, K, dtype, seed):
    counts, align, lead, tail, with_counts = SEGMENTS[seg]
    starts, rows = segments(counts, align, lead, tail)
    off, cnt = device_segments(counts, starts, rows, with_counts)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    x, dy = randn(gen, (rows, K), 1.0, DT[dtype]), randn(gen, (rows, N), 0.5, DT[dtype])
    W = randn(gen, (E, N, K), K ** -0.5, DT[dtype])
    return counts, starts, rows, off, cnt, x, dy, W


def _run(moe, op, x, dy, W, off, cnt, out):
    if op == "mm":
        return moe.moe_grouped_mm(x, W, off, cnt, out=out)
    if op == "dgrad":
        return moe.moe_grouped_dgrad(dy, W, off, cnt, out=out)
    return moe.moe_grouped_wgrad(dy, x, off, cnt, out=out)


def _out(op, rows, E, N, K, dtype):
    shape = {"mm": (rows, N), "dgrad": (rows, K), "wgrad": (E, N, K)}[op]
    return torch.full(shape, SENTINEL, dtype=DT[dtype], device="cuda")


def _verify(op, out, counts, starts, x, dy, W):
    N, K = W.shape[1:]
    live = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for e, (s, n) in enumerate(zip(starts, counts)):
        r = slice(s, s + n)
        live[r] = True
        if op == "mm":
            check(out[r], *mm(x[r], W[e].t()), K, f"mm expert {e}")
        elif op == "dgrad":
            check(out[r], *mm(dy[r], W[e]), N, f"dgrad expert {e}")
        else:
            check(out[e], *mm(dy[r].t(), x[r]), n, f"wgrad expert {e}")
    if op != "wgrad":
        assert (out[~live] == SENTINEL).all(), "rows of no segment were written"


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("seg", SEGMENTS)
def test_segments(moe, op, types, seg):
    N, K = 264, 136
    counts, starts, rows, off, cnt, x, dy, W = _inputs(seg, N, K, types[0], 11)
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, types[1]))
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(op, out, counts, starts, x, dy, W)


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("seg", ["tiles", "few-rows"])
def test_odd_sizes(moe, op, types, size, seg):
    N, K = size
    counts, starts, rows, off, cnt, x, dy, W = _inputs(seg, N, K, types[0], 12)
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, types[1]))
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(op, out, counts, starts, x, dy, W)


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("size", [(4, 12), (12, 4), (132, 4), (4, 1028)], ids=str)
@pytest.mark.parametrize("seg", ["tiles", "few-rows", "padded"])
def test_smallest_steps_fp32(moe, op, size, seg):
    N, K = size
    counts, starts, rows, off, cnt, x, dy, W = _inputs(seg, N, K, "f32", 21)
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, "f32"))
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(op, out, counts, starts, x, dy, W)


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[50, 51, 0, 99, 64, 40], [64], [1, 127], [66, 41, 88], [8, 40, 30]], ids=str)
@pytest.mark.parametrize("size", [(60, 2052), (1100, 60), (64, 64), (44, 396)], ids=str)
def test_middling_segments_fp32(moe, op, counts, size):
    """Rows (for the weight gradient: features) between the heights of two tiles, with and without the
    reduction split."""
    starts, rows = segments(counts, 1, 2, 3)
    off, cnt = device_segments(counts, starts, rows, False)
    gen = torch.Generator(device="cuda").manual_seed(24)
    x, dy = randn(gen, (rows, size[1]), 1.0, DT["f32"]), randn(gen, (rows, size[0]), 0.5, DT["f32"])
    W = randn(gen, (len(counts), *size), size[1] ** -0.5, DT["f32"])
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), *size, "f32"))
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(op, out, counts, starts, x, dy, W)


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[1500, 0, 2600, 900], [9, 8, 0, 7], [60, 200, 2, 90]], ids=str)
@pytest.mark.parametrize("N,K", [(2056, 1736), (5120, 640), (1024, 4608)], ids=str)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_larger(moe, op, counts, N, K, out_dtype):
    """Several waves of tiles, narrow and wide (512 features), few tiles with long reductions."""
    starts, rows = segments(counts)
    off, cnt = device_segments(counts, starts, rows, False)
    gen = torch.Generator(device="cuda").manual_seed(13)
    x, dy = randn(gen, (rows, K), 1.0, DT["bf16"]), randn(gen, (rows, N), 0.5, DT["bf16"])
    W = randn(gen, (len(counts), N, K), K ** -0.5, DT["bf16"])
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, out_dtype))
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(op, out, counts, starts, x, dy, W)
    again = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, out_dtype))
    assert torch.equal(out, again), "not repeatable"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("seg", ["tiles", "few-rows", "padded"])
def test_nan_and_inf_stay_in_their_rows(moe, dtype, seg):
    """NaN and Inf in rows of no segment, or in another expert's rows or weights, reach nothing else."""
    N, K = 136, 200
    counts, starts, rows, off, cnt, x, dy, W = _inputs(seg, N, K, dtype, 14)
    bad = max(range(len(counts)), key=lambda e: counts[e])
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for s, n in zip(starts, counts):
        live[s:s + n] = True
    for t in (x, dy):
        t[~live] = float("nan")
        t[starts[bad]:starts[bad] + counts[bad]] = float("nan")
    W[bad] = float("inf")
    for op in ("mm", "dgrad", "wgrad"):
        out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, dtype))
        for e, (s, n) in enumerate(zip(starts, counts)):
            r = slice(s, s + n)
            got = out[e] if op == "wgrad" else out[r]
            if e == bad:
                assert got.isnan().all()
                continue
            want = {"mm": lambda: (mm(x[r], W[e].t()), K), "dgrad": lambda: (mm(dy[r], W[e]), N),
                    "wgrad": lambda: (mm(dy[r].t(), x[r]), n)}[op]()
            check(got, *want[0], want[1], f"{op} expert {e}")
        if op != "wgrad":
            assert (out[~live] == SENTINEL).all()


def test_one_nan_row_of_a_segment(moe):
    N, K = 128, 64
    counts, starts, rows, off, cnt, x, dy, W = _inputs("tiles", N, K, "bf16", 15)
    row = starts[2] + 200
    x[row, 3] = float("nan")
    y = moe.moe_grouped_mm(x, W, off, cnt)
    assert y[row].isnan().all()
    assert not y[row - 1].isnan().any() and not y[row + 1].isnan().any()
    dW = moe.moe_grouped_wgrad(dy, x, off, cnt)
    assert dW[2, :, 3].isnan().all() and int(dW.isnan().sum()) == N


def test_empty_batch(moe):
    W = torch.ones(4, 16, 24, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    x, dy = W.new_empty(0, 24), W.new_empty(0, 16)
    assert moe.moe_grouped_mm(x, W, off).shape == (0, 16)
    assert moe.moe_grouped_dgrad(dy, W, off).shape == (0, 24)
    dW = moe.moe_grouped_wgrad(dy, x, off, out=W)
    assert (dW == 0).all()


@pytest.mark.parametrize("bad", [[0, 4, 2, 10], [0, 4, 8, 11], [-1, 4, 8, 10]], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_segments_are_reported(moe, bad, dtype):
    """Offsets that decrease or leave the rows, counts that pass the next segment: nothing is written."""
    x = torch.ones(10, 64, dtype=DT[dtype], device="cuda")
    W = torch.ones(3, 64, 64, dtype=DT[dtype], device="cuda")
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for op in ("mm", "dgrad", "wgrad"):
        out = _run(moe, op, x, x, W, off, None, _out(op, 10, 3, 64, 64, dtype))
        assert moe.moe_get_device_status() == moe.MOE_ERR_DEVICE
        assert (out == SENTINEL).all()
    off = torch.tensor([0, 4, 8, 10], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([4, 5, 2], dtype=torch.int32, device="cuda")
    out = _run(moe, "mm", x, x, W, off, cnt, _out("mm", 10, 3, 64, 64, dtype))
    assert moe.moe_get_device_status() == moe.MOE_ERR_DEVICE
    assert (out == SENTINEL).all()


@pytest.mark.parametrize("dtype", ["f32"])
def test_gradients_against_differences(moe, dtype):
    """L = <dy, mm(x, W)> is linear in x and in W: its central difference along a direction v is the inner
    product of the gradient with v up to the rounding of the products (bound of check, summed)."""
    N, K = 72, 104
    counts, starts, rows, off, cnt, x, dy, W = _inputs("mixed", N, K, dtype, 16)
    gen = torch.Generator(device="cuda").manual_seed(17)

    def loss(xx, ww):
        return (moe.moe_grouped_mm(xx, ww, off, cnt).double() * dy.double()).sum().item()

    mag = sum((dy[s:s + n].double().abs() * mm(x[s:s + n], W[e].t())[1]).sum().item()
              for e, (s, n) in enumerate(zip(starts, counts)))
    for grad, t in ((moe.moe_grouped_dgrad(dy, W, off, cnt), x), (moe.moe_grouped_wgrad(dy, x, off, cnt), W)):
        v = randn(gen, t.shape, 1.0, t.dtype) * t.abs()   # |x + v| stays a few |x|
        hi, lo = t + v, t - v
        diff = (loss(hi, W) - loss(lo, W)) if t is x else (loss(x, hi) - loss(x, lo))
        step = (hi.double() - lo.double())                # the step as rounded
        want = (grad.double() * step).sum().item()
        # three results, each within (n + 8 + 1) 2^-23 of magnitudes at most 6 times those at x
        bound = 3 * (max(N, K, rows) + 9) * 2.0 ** -23 * 6 * mag
        assert abs(diff - want) <= bound, (diff, want, bound)


def test_other_stream_and_graph(moe):
    N, K = 512, 256
    counts, starts, rows, off, cnt, x, dy, W = _inputs("tiles", N, K, "bf16", 18)
    ref = [_run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, "bf16"))
           for op in ("mm", "dgrad", "wgrad")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [_out(op, rows, len(counts), N, K, "bf16") for op in ("mm", "dgrad", "wgrad")]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for op, o in zip(("mm", "dgrad", "wgrad"), got):
            _run(moe, op, x, dy, W, off, cnt, o)
    side.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    # captured: the offsets, rows and weights are read at replay
    g = torch.cuda.CUDAGraph()
    for o in got:
        o.fill_(SENTINEL)
    with torch.cuda.graph(g):
        for op, o in zip(("mm", "dgrad", "wgrad"), got):
            _run(moe, op, x, dy, W, off, cnt, o)
    new_counts = [9, 200, 100, 0, 300, 97]
    assert sum(new_counts) == sum(counts)
    new_starts, _ = segments(new_counts, 1, 3, 9)
    off.copy_(torch.tensor(new_starts + [rows], dtype=torch.int32))
    cnt.copy_(torch.tensor(new_counts, dtype=torch.int32))
    x.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    for op, o in zip(("mm", "dgrad", "wgrad"), got):
        _verify(op, o, new_counts, new_starts, x, dy, W)
    assert moe.moe_get_device_status() == moe.MOE_OK


def test_concurrent_calls_on_two_streams(moe):
    N, K = 1032, 776
    counts, starts, rows, off, cnt, x, dy, W = _inputs("long", N, K, "bf16", 19)
    ref = moe.moe_grouped_mm(x, W, off, cnt)
    refd = moe.moe_grouped_dgrad(dy, W, off, cnt)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(ref), torch.empty_like(refd)] for _ in range(6)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(outs):
        with torch.cuda.stream(streams[i % 2]):
            moe.moe_grouped_mm(x, W, off, cnt, out=a)
            moe.moe_grouped_dgrad(dy, W, off, cnt, out=b)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == moe.MOE_OK
    for a, b in outs:
        assert torch.equal(a, ref) and torch.equal(b, refd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_outputs_past_32_bit_offsets(moe, op, dtype):
    """More than 2^31 output elements: the last rows (and the first) are right."""
    small, big = 64, 2 ** 31 // 40000 + 3000
    rows, N, K = {"mm": (big, 40000, small), "dgrad": (big, small, 40000), "wgrad": (7, 40000, big // 8 * 8)}[op]
    gen = torch.Generator(device="cuda").manual_seed(20)
    counts = [rows - 3, 3]
    starts, _ = segments(counts)
    off, _ = device_segments(counts, starts, rows, False)
    x = randn(gen, (rows, K), 1.0, DT[dtype]) if op != "dgrad" else None
    dy = randn(gen, (rows, N), 1.0, DT[dtype]) if op != "mm" else None
    W = randn(gen, (2, N, K), 0.1, DT[dtype]) if op != "wgrad" else None
    out = _run(moe, op, x, dy, W, off, None, None)
    assert out.numel() > 2 ** 31
    assert moe.moe_get_device_status() == moe.MOE_OK
    for e, (s, n) in enumerate(zip(starts, counts)):
        for part in (slice(0, 64), slice(-64, None)):
            r = torch.arange(s, s + n, device="cuda")[part]
            if op == "mm":
                check(out[r], *mm(x[r], W[e].t()), K, "mm")
            elif op == "dgrad":
                check(out[r], *mm(dy[r], W[e]), N, "dgrad")
            else:
                check(out[e][part], *mm(dy[s:s + n, part].t(), x[s:s + n]), n, "wgrad")


def test_with_the_layers_dispatch(moe):
    """route -> dispatch -> grouped products -> combine is the layer: equal to moe_forward up to the bf16
    rounding of the pre-activations and of the expert outputs, which the fused layer keeps in fp32."""
    import moe_inputs
    from moe_testlib import upload
    T, d, F, E, k = 300, 256, 512, 8, 2
    x, Wg, W1, W3, W2 = upload(moe_inputs.make_inputs(T, d, F, E, k, "bf16", seed=31))
    idx, w = moe.moe_route(x, Wg, k)
    counts, offsets, perm, inv = moe.moe_dispatch(idx, E)
    rows = moe.moe_slots_capacity(T, E, k)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    live[inv.reshape(-1).long()] = True
    xp = torch.full((rows, d), float("nan"), dtype=x.dtype, device="cuda")
    xp[live] = x[(perm[live] // k).long()]
    a = moe.moe_grouped_mm(xp, W1, offsets, counts, out_dtype=torch.float32)
    b = moe.moe_grouped_mm(xp, W3, offsets, counts, out_dtype=torch.float32)
    h = torch.zeros(rows, F, dtype=x.dtype, device="cuda")
    h[live] = (torch.nn.functional.silu(a[live]) * b[live]).to(x.dtype)
    y = moe.moe_grouped_mm(h, W2, offsets, counts, out_dtype=torch.float32)
    out = (y[inv.long()] * w[..., None]).sum(1)
    ref = moe.moe_forward(x, Wg, W1, W3, W2, k).float()
    assert moe.moe_get_device_status() == moe.MOE_OK
    # h: equal fp32 pre-activations up to summation order and the fast exponential, then one bf16 rounding
    # that may fall the other way (2^-7 of a term); the output's own rounding 2^-8
    mag = torch.zeros(T, d, device="cuda", dtype=torch.float64)
    for e in range(E):
        s, n = int(offsets[e]), int(counts[e])
        ym = h[s:s + n].double().abs() @ W2[e].double().abs().t()
        tok = (perm[s:s + n] // k).long()
        slot = (perm[s:s + n] % k).long()
        mag.index_add_(0, tok, ym * w[tok, slot].double()[:, None])
    bound = (2.0 ** -7 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.double().abs()
    assert ((out.double() - ref.double()).abs() <= bound).all()
