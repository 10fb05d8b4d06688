"""The kernels that only some sizes reach: weight gradients with a split reduction and on 512-feature tiles, the
16-row few-row kernel; and how far fp32 results are off at long reductions."""
import pytest
import torch

from grouped_testlib import DT, device_segments, randn, segments
from test_gpu_grouped import _out, _run, _verify
from test_gpu_lora import _call, _inputs
from test_gpu_lora import _verify as _verify_lora

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


def _product(moe, op, counts, N, K, types, seed, align=1):
    starts, rows = segments(counts, align, 0, 0)
    off, cnt = device_segments(counts, starts, rows, align > 1)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = randn(gen, (rows, K), 1.0, DT[types[0]]), randn(gen, (rows, N), 0.5, DT[types[0]])
    W = randn(gen, (len(counts), N, K), K ** -0.5, DT[types[0]])
    out = _run(moe, op, x, dy, W, off, cnt, _out(op, rows, len(counts), N, K, types[1]))
    assert moe.moe_get_device_status() == moe.MOE_OK
    return out, starts, x, dy, W


@pytest.mark.parametrize("counts", [[1500, 900], [2050, 0, 1031], [4097], [1, 3000, 600]], ids=str)
@pytest.mark.parametrize("size", [(264, 264), (72, 520), (520, 136)], ids=str)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_wgrad_with_a_split_reduction(moe, counts, size, out_dtype):
    """Few tiles and at least 512 rows to a segment on average; segments of any length, or empty."""
    out, starts, x, dy, W = _product(moe, "wgrad", counts, *size, ("bf16", out_dtype), 51)
    _verify("wgrad", out, counts, starts, x, dy, W)


@pytest.mark.parametrize("counts", [[300, 0, 130, 77, 90], [1000, 3, 0, 64, 400]], ids=str)
def test_wgrad_on_wide_tiles(moe, counts):
    """bf16 output, 5 x 16 x 9 tiles of half the size: at least two waves of 512-feature ones."""
    N, K = 1024, 4608
    out, starts, x, dy, W = _product(moe, "wgrad", counts, N, K, ("bf16", "bf16"), 52)
    _verify("wgrad", out, counts, starts, x, dy, W)


@pytest.mark.parametrize("rows", [17, 24, 31, 32])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(328, 264), (40, 2056)], ids=str)
def test_few_rows_of_one_expert(moe, rows, out_dtype, size):
    out, starts, x, dy, W = _product(moe, "mm", [rows], *size, ("bf16", out_dtype), 53)
    _verify("mm", out, [rows], starts, x, dy, W)


@pytest.mark.parametrize("rows", [17, 24, 32])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["random", "each"])
@pytest.mark.parametrize("R", [8, 64])
def test_few_rows_of_one_expert_with_adapters(moe, rows, out_dtype, pattern, R):
    N, K, L = 328, 520, 5
    a = _inputs([rows], N, K, L, R, pattern, 54)
    out = _call(moe, [rows], a[0], a[1], False, out_dtype, *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify_lora(out, [rows], a[0], *a[2:])


# How far a long sum of random terms may be off, RMS of the error over RMS of the result, in units of 2^-23.  An
# addition of a term to a running sum s that rounds to nearest errs by ulp(s) / sqrt(12), on average over s's mantissa
# 0.21 2^-23 |s| (RMS); one that truncates, as the tensor cores do, by half an ulp in one direction, 0.36 2^-23 |s|.
# With |s| = sqrt(k) of k terms of unit size:
#   rounded, one chain of n:            0.21 sqrt(n / 2)                                        (n = 14336: 17.8)
#   truncated, 16 terms to an addition, m additions to an accumulator, accumulators added with rounding:
#       0.36 (4 * 2/3 m^1.5) / sqrt(16 m) = 0.24 m, and the rounded additions of n / 16 m sums   (m = 32: 7.7)
N_LONG = 14336
TILE, FEW, SIMT, ADAPTERS = 8.0, 3.0, 18.0, 9.0   # m = 32; m = 8; one chain of them all; m = 32 and u's own sums


def _rms_error(got, want):
    return ((got.double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()).item() * 2.0 ** 23


@pytest.mark.parametrize("dtype,op,counts,N,limit", [
    ("bf16", "mm", [2000, 1800], 2048, TILE), ("bf16", "mm", [200], 264, TILE), ("bf16", "mm", [3, 40, 300], 264, TILE),
    ("bf16", "mm", [8], 1024, FEW), ("bf16", "mm", [24], 520, FEW), ("bf16", "mm", [5, 0, 7, 9], 520, FEW),
    ("bf16", "dgrad", [900, 1100], 520, TILE), ("bf16", "wgrad", [N_LONG], 512, TILE),
    ("bf16", "wgrad", [N_LONG, 100], 2048, TILE),
    ("f32", "mm", [2000, 1800], 2048, SIMT), ("f32", "mm", [60], 512, SIMT), ("f32", "mm", [30, 30, 25, 9], 512, SIMT),
    ("f32", "mm", [7], 512, SIMT), ("f32", "dgrad", [300], 520, SIMT), ("f32", "wgrad", [N_LONG], 1024, SIMT),
], ids=str)
def test_long_sums_in_fp32(moe, dtype, op, counts, N, limit):
    """Reductions of 14336 into fp32: what blocked accumulators and split sums are for."""
    K = 768 if op == "wgrad" else N_LONG
    size = (N_LONG, N) if op == "dgrad" else (N, K)
    out, starts, x, dy, W = _product(moe, op, counts, *size, (dtype, "f32"), 55)
    for e, (s, n) in enumerate(zip(starts, counts)):
        r = slice(s, s + n)
        if n == 0 or (op == "wgrad" and n < N_LONG):
            continue
        a, b, got = {"mm": lambda: (x[r], W[e].t(), out[r]), "dgrad": lambda: (dy[r], W[e], out[r]),
                     "wgrad": lambda: (dy[r].t(), x[r], out[e])}[op]()
        err = _rms_error(got, a.double() @ b.double())
        assert err <= limit, (e, err, limit)


@pytest.mark.parametrize("counts,limit", [([2000], ADAPTERS), ([200], ADAPTERS), ([8], FEW + 1), ([30], FEW + 1)], ids=str)
def test_long_sums_in_fp32_with_adapters(moe, counts, limit):
    N, L, R = 520, 5, 64
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, N, N_LONG, L, R, "runs", 56)
    out = _call(moe, counts, starts, rows, False, "f32", x, W, A, B, scale, ids)
    want = x.double() @ W[0].double().t()
    for a in range(L):
        m = ids == a
        want[m] += (x[m].double() @ A[a, 0].double().t() * scale[a].double()) @ B[a, 0].double().t()
    err = _rms_error(out, want)
    assert err <= limit, (err, limit)


@pytest.mark.parametrize("counts", [[2, 0, 5, 1], [29]], ids=str)
@pytest.mark.parametrize("R", [8, 64])
def test_few_rows_with_adapters_are_rounded_once(moe, counts, R):
    """bf16 outputs of batches of few rows: s A x keeps 16 bits, so the output's own rounding is all there is.  RMS
    errors: the rounding alone is about 1.7e-3 of the result; u is off by 2^-16 and the fp32 sums by 1e-6 at most,
    which add a ten-thousandth to it (u in one bf16 value: a tenth)."""
    N, K, L = 520, 1032, 4
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, N, K, L, R, "each", 57)
    out = _call(moe, counts, starts, rows, False, "bf16", x, W, A, B, scale, ids)
    want = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    for e, (s, n) in enumerate(zip(starts, counts)):
        for r in range(s, s + n):
            a, xr = int(ids[r]), x[r].double()
            want[r] = W[e].double() @ xr + B[a, e].double() @ (scale[a].double() * (A[a, e].double() @ xr))
    rms = lambda t: t.double().pow(2).mean().sqrt().item()
    assert rms(out.double() - want) <= 1.001 * rms(want.bfloat16().double() - want)


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per", [1, 20])
def test_adapters_of_256_experts(moe, out_dtype, per):
    counts = [per if e % 3 else 0 for e in range(256)]
    a = _inputs(counts, 72, 136, 3, 8, "random", 58, lead=1, tail=2)
    out = _call(moe, counts, a[0], a[1], True, out_dtype, *a[2:])
    assert moe.moe_get_device_status() == moe.MOE_OK
    _verify_lora(out, counts, a[0], *a[2:])


def test_adapters_of_an_empty_batch(moe):
    bf = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = moe.moe_grouped_lora(bf(0, 64), bf(2, 40, 64), off, bf(4, 2, 8, 64), bf(4, 2, 40, 8),
                               torch.ones(4, device="cuda"), off[:0])
    assert out.shape == (0, 40) and moe.moe_get_device_status() == moe.MOE_OK
