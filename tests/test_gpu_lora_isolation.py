"""A non-finite adapter reaches its own rows only, in every kernel that multiplies a tile's adapters together
(narrow, wide, split; both output types), and does not hold up the other requests of its batch."""
import pytest
import torch

from grouped_testlib import DT, device_segments
from test_gpu_lora import _call, _inputs, _verify

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


# counts, N, K: narrow tiles, several to a pair of CTAs; tiles split over pairs; 512-feature tiles (bf16
# output); few rows of padded segments beside long ones
SIZES = {
    "narrow": ([900, 0, 1500], 1800, 200),
    "split": ([290], 136, 2048),
    "split-two": ([130, 45], 264, 1032),
    "wide": ([2500, 700, 1, 1800], 5120, 328),
    "mixed": ([12, 130, 0, 40], 520, 264),
}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pattern", ["random", "runs"])
@pytest.mark.parametrize("bad", ["factor", "feature", "rows"])
def test_other_rows_keep_their_values(moe, size, out_dtype, pattern, bad):
    """B of one adapter infinite throughout, or NaN in one feature of one expert; A NaN (its rows of u)."""
    counts, N, K = SIZES[size]
    L, R = 7, 32
    with_counts = size == "mixed"
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, N, K, L, R, pattern, 71, align=128 if with_counts else 1)
    hit = ids == 3
    if bad == "factor":
        B[3] = float("inf")
    elif bad == "feature":
        B[3, 0, N // 2 + 1] = float("nan")
    else:
        A[3] = float("nan")
    out = _call(moe, counts, starts, rows, with_counts, out_dtype, x, W, A, B, scale, ids)
    assert moe.moe_get_device_status() == moe.MOE_OK
    # the bad adapter's own rows: what the formula gives; the others as if it were not there
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for s, n in zip(starts, counts):
        live[s:s + n] = True
    mine = hit & live
    first = torch.zeros_like(live)
    first[starts[0]:starts[0] + counts[0]] = True
    if bad == "factor":
        assert not out[mine].isfinite().any()
        again = mine
    elif bad == "feature":
        assert out[mine & first, N // 2 + 1].isnan().all()
        again = mine
        ok = torch.ones(N, dtype=torch.bool, device="cuda")
        ok[N // 2 + 1] = False
        assert out[mine][:, ok].isfinite().all()
    else:
        assert out[mine].isnan().all()
        again = mine
    clean = torch.where(hit, torch.full_like(ids, -1), ids)
    A[3], B[3] = 0, 0
    out[again] = _call(moe, counts, starts, rows, with_counts, out_dtype, x, W, A, B, scale, clean)[again]
    _verify(out, counts, starts, x, W, A, B, scale, clean)


def _time(f, n):
    f()
    torch.cuda.synchronize()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    for _ in range(n):
        f()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / n


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_a_bad_adapter_does_not_hold_up_the_batch(moe, out_dtype):
    """Every output of the batch is touched by the bad adapter's products.  A clean call is tens of
    microseconds; with the outputs summed again from global memory at a hundredth of the tensor cores' rate it may
    take 100 times that, not thousands."""
    counts, N, K, L, R = [1500], 2048, 2048, 7, 32
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, N, K, L, R, "runs", 72)
    off, _ = device_segments(counts, starts, rows, False)
    out = torch.empty(rows, N, dtype=DT[out_dtype], device="cuda")
    call = lambda: moe.moe_grouped_lora(x, W, off, A, B, scale, ids, out=out)
    clean = _time(call, 20)
    B[3] = float("inf")
    slow = _time(call, 2)
    print(f"clean {clean * 1e3:.1f} us, with an infinite adapter {slow * 1e3:.1f} us")
    assert moe.moe_get_device_status() == moe.MOE_OK
    assert slow <= 100 * clean, (clean, slow)


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_long_reductions_with_a_bad_adapter(moe, out_dtype):
    """Several tiles to a pair of CTAs, every output of each to be summed again over a reduction of 57344: no
    bounded wait of the pipeline may run out meanwhile."""
    counts, N, K, L, R = [2048], 4096, 57344, 5, 16
    starts, rows, x, W, A, B, scale, ids = _inputs(counts, N, K, L, R, "runs", 73)
    B[2] = float("inf")
    out = _call(moe, counts, starts, rows, False, out_dtype, x, W, A, B, scale, ids)
    assert moe.moe_get_device_status() == moe.MOE_OK
    hit = ids == 2
    assert not out[hit].isfinite().any()
    clean = torch.where(hit, torch.full_like(ids, -1), ids)
    B[2] = 0
    out[hit] = _call(moe, counts, starts, rows, False, out_dtype, x, W, A, B, scale, clean)[hit]
    _verify(out, counts, starts, x, W, A, B, scale, clean)
