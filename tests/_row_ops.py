"""Inputs and error bounds shared by the tests of the row-wise operators.

Bounds are |got - ref| <= U[dtype] |ref| + TINY[dtype] + (an fp32 part), ref in fp64. U is half a unit in
the last place, the one rounding of an output. The fp32 part comes from the arithmetic: SUM = 2^-17 for a
sum (a thread adds at most some 100 terms in sequence, in pairs or lanes, before a tree of at most 10
levels: (100 + 10) 2^-24 < 2^-17) relative to the sum of the terms' magnitudes, and EXP = 2^-21 for an
exponential's own error (ex2.approx: 2 ulp, and the scaled argument's rounding, 2^-23 of its size, is
added by the caller).
"""

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
SUM = 2.0 ** -17
EXP = 2.0 ** -21
NAME = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
DTYPES = list(NAME)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, ref, dtype, fp32_part):
    """got (a tensor) against ref (fp64, any non-finite values equal) within the bound."""
    g = f64(got).reshape(np.shape(ref))
    ref = np.asarray(ref, np.float64)
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(np.isnan(g), np.isnan(ref), err_msg=name)
    inf = np.isinf(ref)
    np.testing.assert_array_equal(g[inf], ref[inf], err_msg=name)
    bound = U[dtype] * np.abs(ref) + TINY[dtype] + np.broadcast_to(fp32_part, ref.shape)
    with np.errstate(invalid="ignore"):
        bad = fine & ~(np.abs(g - ref) <= bound)
    if bad.any():
        i = np.argwhere(bad)[0]
        raise AssertionError(f"{name}: {int(bad.sum())} of {ref.size} outside the bound, first at {tuple(i)}: "
                             f"got {g[tuple(i)]!r}, ref {ref[tuple(i)]!r}, bound {bound[tuple(i)]:.3g}")


def strided(t, layout):
    """t's values in another layout: "dense", "padded" rows, rows starting one element into a buffer
    ("shifted", misaligned for vectors), "transposed" (elements of a row far apart)."""
    M, N = t.shape
    if layout == "dense":
        return t.contiguous()
    if layout == "padded":
        pad = 8 if N % 8 == 0 else 3
        b = torch.full((M, N + pad), float("nan"), dtype=t.dtype, device=t.device)
        b[:, :N] = t
        return b[:, :N]
    if layout == "shifted":
        b = torch.full((M * N + 1,), float("nan"), dtype=t.dtype, device=t.device)
        b[1:] = t.reshape(-1)
        return b[1:].view(M, N)
    if layout == "transposed":
        return t.t().contiguous().t()
    raise ValueError(layout)


LAYOUTS = ("dense", "padded", "shifted", "transposed")
