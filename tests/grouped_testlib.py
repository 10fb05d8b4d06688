"""Segments, inputs, 64-bit references and error bounds for the tests of the grouped products.

Bounds (per element, worst case).  Inputs are exact.  A product sum over n terms in fp32 is off by
at most (n + 8) 2^-23 sum |terms| whatever its order (one rounding of up to an ulp, 2^-23, per
addition: the tensor cores may truncate where the CUDA cores round); the result's own rounding adds
eps/2 of the value, a bf16 intermediate eps/2 of its own.
"""
from __future__ import annotations

import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U32 = 2.0 ** -23


def half_ulp(dtype):
    return torch.finfo(dtype).eps / 2


def segments(counts, align=1, lead=0, tail=0):
    """(starts, rows of the buffers) of segments of the given row counts."""
    starts, row = [], lead
    for n in counts:
        starts.append(row)
        row += -(-n // align) * align
    return starts, row + tail


def device_segments(counts, starts, rows, with_counts):
    off = torch.tensor(starts + [rows], dtype=torch.int32, device="cuda")
    if not with_counts:   # the last segment then has to end at offsets[E]
        off[-1] = starts[-1] + counts[-1]
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda") if with_counts else None
    return off, cnt


def randn(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def mm(a, b):
    """a @ b in 64 bits and the same of the magnitudes."""
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def check(got, want, mag, n, what, extra=0.0):
    """|got - want| within the bound for a sum of n terms of total magnitude mag (and extra)."""
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = (n + 8) * U32 * mag + half_ulp(got.dtype) * want.abs() * (1 + 1e-3) + extra + 1e-37
    excess = ((got.double() - want).abs() / bound).max().item() if got.numel() else 0.0
    assert excess <= 1.0, f"{what}: error {excess:.2f} times its bound"
