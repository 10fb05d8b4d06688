"""Bad segment tables of which no segment has rows: recorded, and nothing is written."""
import pytest
import torch

from grouped_testlib import DT
from test_gpu_grouped import SENTINEL, _out, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import sparse_mixture_experts_14_b200 as m
    return m


@pytest.mark.parametrize("offsets,counts", [([5, 3], None), ([4, 2, 2], None), ([0, 11], None), ([0, 4], [5]),
                                            ([-1, 0, 0], None), ([0, 4, 4], [-1, 0])], ids=str)
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
def test_bad_tables_without_rows(moe, op, types, offsets, counts):
    E = len(offsets) - 1
    x = torch.ones(10, 64, dtype=DT[types[0]], device="cuda")
    W = torch.ones(E, 64, 64, dtype=DT[types[0]], device="cuda")
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = _run(moe, op, x, x, W, off, cnt, _out(op, 10, E, 64, 64, types[1]))
    assert moe.moe_get_device_status() == moe.MOE_ERR_DEVICE
    assert (out == SENTINEL).all()
