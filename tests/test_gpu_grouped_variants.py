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
