"""moe_grouped_lora against y_r = W_e x_r + B_{a,e} (s_a A_{a,e} x_r) in 64 bits: every rank, adapters in
runs and at random, rows without one, many in one tile, few rows and many, bad ids, graphs."""
import pytest
import torch

from grouped_testlib import DT, U32, check, device_segments, half_ulp, mm, randn, segments

pytestmark = pytest.mark.gpu

SENTINEL = -77.0


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


def _inputs(counts, N, K, L, R, pattern, seed, lead=0, tail=0, align=1):
    starts, rows = segments(counts, align, lead, tail)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    x = randn(gen, (rows, K), 1.0, DT["bf16"])
    W = randn(gen, (E, N, K), K ** -0.5, DT["bf16"])
    A = randn(gen, (L, E, R, K), K ** -0.5, DT["bf16"])
    B = randn(gen, (L, E, N, R), R ** -0.5, DT["bf16"])
    scale = torch.rand(L, generator=gen, device="cuda") * 2 - 0.5
    r = torch.arange(rows, device="cuda")
    ids = {"random": torch.randint(-1, L, (rows,), generator=gen, device="cuda"), "runs": (r // 37) % (L + 1) - 1,
           "none": torch.full_like(r, -1), "one": torch.full_like(r, L - 1),
           "each": r % L, "alternate": torch.where(r % 2 == 0, r % L, torch.full_like(r, -1))}[pattern]
    return starts, rows, x, W, A, B, scale, ids.int()


def _verify(out, counts, starts, x, W, A, B, scale, ids):
    N, K = W.shape[1:]
    R = A.shape[2]
    live = torch.zeros(x.shape[0], dtype=torch.bool, device="cuda")
    for e, (s, n) in enumerate(zip(starts, counts)):
        r = slice(s, s + n)
        live[r] = True
        want, mag = mm(x[r], W[e].t())
        extra = torch.zeros_like(want)
        for a in ids[r].unique().tolist():
            if a < 0:
                continue
            mine = (ids[r] == a).nonzero()[:, 0]
            u, um = mm(x[r][mine] , A[a, e].t())
            u, um = u * scale[a].double(), um * scale[a].double().abs()
            want[mine] += u @ B[a, e].double().t()
            # u as it is used: its own sum, then one rounding to bf16, or to fp32's 24 bits beside an fp32 output
            uerr = (K + 9) * U32 * um + half_ulp(out.dtype) * u.abs() * (1 + 1e-3)
            babs = B[a, e].double().abs().t()
            extra[mine] += (1 + 1e-3) * uerr @ babs
            mag[mine] += u.abs() @ babs
        check(out[r], want, mag, K + R, f"expert {e}", extra)
    assert (out[~live] == SENTINEL).all(), "rows of no segment were written"


def _call(moe, counts, starts, rows, with_counts, out_dtype, x, W, A, B, scale, ids):
    off, cnt = device_segments(counts, starts, rows, with_counts)
    out = torch.full((rows, W.shape[1]), SENTINEL, dtype=DT[out_dtype], device="cuda")
    return moe.moe_grouped_lora(x, W, off, A, B, scale, ids, counts=cnt, out=out)


@pytest.mark.parametrize("R", [8, 16, 24, 64, 104, 128])
@pytest.mark.parametrize("pattern", ["random", "runs"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[3, 0, 2, 9], [300, 1, 0, 70], [40, 60, 33, 2]], ids=str)
def test_ranks(moe, R, pattern, out_dtype, counts):
    N, K, L = 328, 264, 5
    a = _inputs(counts, N, K, L, R, pattern, R)
    out = _call(moe, counts, a[0], a[1], False, out_dtype, *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(out, counts, a[0], *a[2:])


@pytest.mark.parametrize("pattern", ["none", "one", "each", "alternate", "random"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[1], [6, 0, 5], [290, 0, 31]], ids=str)
def test_patterns(moe, pattern, out_dtype, counts):
    """Up to a different adapter for every row of a tile."""
    N, K, L, R = 136, 520, 260, 16
    a = _inputs(counts, N, K, L, R, pattern, 5, lead=2, tail=7)
    out = _call(moe, counts, a[0], a[1], True, out_dtype, *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(out, counts, a[0], *a[2:])


@pytest.mark.parametrize("size", [(8, 8), (2056, 40), (520, 2048)], ids=str)
@pytest.mark.parametrize("counts", [[2, 1], [130, 7]], ids=str)
def test_sizes(moe, size, counts):
    N, K = size
    a = _inputs(counts, N, K, 3, 32, "random", 6)
    out = _call(moe, counts, a[0], a[1], False, "f32", *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(out, counts, a[0], *a[2:])


@pytest.mark.parametrize("counts", [[2000], [900, 0, 1500], [2500, 700, 1, 1800]], ids=str)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1032, 904), (5120, 328)], ids=str)
def test_larger(moe, counts, out_dtype, N, K):
    """Several waves of tiles, narrow and wide, and tiles split over pairs."""
    L, R = 7, 64
    a = _inputs(counts, N, K, L, R, "runs", 7)
    out = _call(moe, counts, a[0], a[1], False, out_dtype, *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify(out, counts, a[0], *a[2:])
    assert torch.equal(out, _call(moe, counts, a[0], a[1], False, out_dtype, *a[2:])), "not repeatable"


@pytest.mark.parametrize("counts", [[3, 4], [200, 100]], ids=str)
def test_without_adapters_it_is_the_grouped_product(moe, counts):
    a = _inputs(counts, 264, 136, 4, 16, "none", 8)
    off, cnt = device_segments(counts, a[0], a[1], False)
    x, W, A, B, scale, ids = a[2:]
    A.fill_(float("nan"))
    B.fill_(float("inf"))
    assert torch.equal(moe.moe_grouped_lora(x, W, off, A, B, scale, ids), moe.moe_grouped_mm(x, W, off))


@pytest.mark.parametrize("counts", [[9], [290]], ids=str)
def test_adapters_stay_apart(moe, counts):
    """NaN in one adapter, Inf in another's factor, reach their own rows only."""
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, 136, 264, 4, 16, "each", 9)
    A[1] = float("nan")
    B[2] = float("inf")
    off, _ = device_segments(counts, starts, rows, False)
    out = moe.moe_grouped_lora(x, W, off, A, B, scale, ids)
    assert out[ids == 1].isnan().all()
    assert not out[ids == 2].isfinite().any()
    keep = (ids == 0) | (ids == 3)
    assert out[keep].isfinite().all()
    # The kept rows hold their own terms alone.  Not compared bit for bit with a clean batch: where a
    # neighbour's infinity meets a zero in the tensor cores' sum, the output is summed again in another
    # order.  Either order is within check's bound of the exact value: n + 8 roundings of at most an ulp.
    ids = torch.where(keep, ids, torch.full_like(ids, -1))
    A[1], B[2] = 0, 0
    out[~keep] = moe.moe_grouped_lora(x, W, off, A, B, scale, ids)[~keep]
    _verify(out, counts, starts, x, W, A, B, scale, ids)


@pytest.mark.parametrize("counts", [[5, 4], [200, 90]], ids=str)
@pytest.mark.parametrize("bad", [-2, 4, 2 ** 31 - 1])
def test_bad_ids_are_reported(moe, counts, bad):
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, 64, 64, 4, 8, "random", 10, tail=3)
    ids[-1] = bad   # a row of no segment: not looked at
    _call(moe, counts, starts, rows, True, "bf16", x, W, A, B, scale, ids)
    assert moe.moe_get_device_status() == moe.MOE_OK
    ids[2] = bad
    _call(moe, counts, starts, rows, True, "bf16", x, W, A, B, scale, ids)
    assert moe.moe_get_device_status() == moe.MOE_ERR_DEVICE


@pytest.mark.parametrize("counts", [[7, 0, 6], [200, 0, 90]], ids=str)
def test_graph_reads_ids_at_replay(moe, counts):
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, 264, 136, 6, 16, "runs", 11)
    off, cnt = device_segments(counts, starts, rows, True)
    ws = torch.empty(moe.moe_grouped_lora_workspace_size(rows, 3, 6, 16), dtype=torch.uint8, device="cuda")
    out = torch.full((rows, 264), SENTINEL, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_lora(x, W, off, A, B, scale, ids, counts=cnt, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_grouped_lora(x, W, off, A, B, scale, ids, counts=cnt, out=out, workspace=ws)
    ids.copy_(torch.randint(-1, 6, (rows,), device="cuda", dtype=torch.int32))
    x.neg_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    _verify(out, counts, starts, x, W, A, B, scale, ids)
    assert moe.moe_get_device_status() == moe.MOE_OK


@pytest.mark.parametrize("counts", [[5, 4], [300, 90]], ids=str)
def test_inputs_written_just_before_the_call(moe, counts):
    """Rows, ids, offsets and weights that kernels still in flight write: the call's kernels start early and
    must wait for them."""
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, 776, 520, 6, 32, "random", 13)
    off, _ = device_segments(counts, starts, rows, False)
    big = torch.randn(4096, 4096, device="cuda")
    want = moe.moe_grouped_lora(x, W, off, A, B, scale, ids)
    live = [torch.zeros_like(t) for t in (x, W, off, A, B, scale, ids)]
    for i in range(6):
        for t in live:
            t.zero_()
        out = torch.full_like(want, SENTINEL)
        torch.cuda.synchronize()
        busy = big @ big   # something to wait behind
        for t, v in zip(live, (x, W, off, A, B, scale, ids)):
            t.copy_(v)
        lx, lW, loff, lA, lB, lscale, lids = live
        moe.moe_grouped_lora(lx, lW, loff, lA, lB, lscale, lids, out=out)
        lx.zero_()         # and nothing after the call is too early
        lB.zero_()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    assert moe.moe_get_device_status() == moe.MOE_OK and torch.isfinite(busy).all()


@pytest.mark.parametrize("counts", [[5, 4], [300, 90]], ids=str)
def test_two_calls_at_once(moe, counts):
    """On two streams, with scratch of their own (the binding's, allocated on the stream of the call)."""
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, 776, 520, 6, 32, "random", 12)
    off, _ = device_segments(counts, starts, rows, False)
    ids2 = ids.flip(0).contiguous()
    refs = [moe.moe_grouped_lora(x, W, off, A, B, scale, i) for i in (ids, ids2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[moe.moe_grouped_lora(x, W, off, A, B, scale, i, stream=s) for i, s in zip((ids, ids2), streams)]
            for _ in range(8)]
    torch.cuda.synchronize()
    assert moe.moe_get_device_status() == moe.MOE_OK
    for pair in outs:
        assert torch.equal(pair[0], refs[0]) and torch.equal(pair[1], refs[1])


def test_adapters_on_the_layers_experts(moe):
    """A served batch: route, dispatch, adapters of every request on all three expert matrices, combine."""
    import moe_inputs
    from moe_testlib import upload
    T, d, F, E, k, L, R = 40, 256, 512, 8, 2, 6, 16
    x, Wg, W1, W3, W2 = upload(moe_inputs.make_inputs(T, d, F, E, k, "bf16", seed=33))
    gen = torch.Generator(device="cuda").manual_seed(34)
    ab = [(randn(gen, (L, E, R, K), K ** -0.5, DT["bf16"]), randn(gen, (L, E, N, R), R ** -0.5, DT["bf16"]))
          for N, K in ((F, d), (F, d), (d, F))]
    scale = torch.full((L,), 0.5, device="cuda")
    request = torch.randint(-1, L, (T,), generator=gen, device="cuda", dtype=torch.int32)
    idx, w = moe.moe_route(x, Wg, k)
    counts, offsets, perm, inv = moe.moe_dispatch(idx, E)
    rows = moe.moe_slots_capacity(T, E, k)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    live[inv.reshape(-1).long()] = True
    tok = torch.zeros(rows, dtype=torch.long, device="cuda")
    tok[live] = (perm[live] // k).long()
    ids = torch.where(live, request[tok], torch.full_like(request[tok], 99))
    xp = x[tok].contiguous()

    def lora(rows_in, W, m):
        return moe.moe_grouped_lora(rows_in, W, offsets, *ab[m], scale, ids, counts=counts, out_dtype=torch.float32)

    h = (torch.nn.functional.silu(lora(xp, W1, 0)) * lora(xp, W3, 1)).to(x.dtype)
    h[~live] = 0
    y = lora(h, W2, 2)
    out = (y[inv.long()] * w[..., None]).sum(1)
    assert moe.moe_get_device_status() == moe.MOE_OK
    want, mag = torch.zeros(T, d, dtype=torch.float64), torch.zeros(T, d, dtype=torch.float64)
    f64 = lambda t: t.double().cpu()
    for t in range(T):
        for j in range(k):
            e, a, g = int(idx[t, j]), int(request[t]), float(w[t, j])
            eff = [f64(W[e]) + (0.5 * f64(ab[m][1][a, e]) @ f64(ab[m][0][a, e]) if a >= 0 else 0)
                   for m, W in enumerate((W1, W3, W2))]
            xt = f64(x[t])
            p, q = eff[0] @ xt, eff[1] @ xt
            ht = p * torch.sigmoid(p) * q
            want[t] += g * (eff[2] @ ht)
            mag[t] += g * (eff[2].abs() @ ht.abs())
    # the bf16 roundings of u (twice) and of h, as in the layer's own tolerance: 2e-2 of the output's RMS
    err = (out.double().cpu() - want).abs().max().item()
    assert err <= 2e-2 * mag.pow(2).mean().sqrt().item()
