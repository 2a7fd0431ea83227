"""Inputs, float64 values and error bounds for the feed-forward GPU tests.

Bounds count what the kernels do.  U = 2^-24 is half a float32 step, and a
float32 sum of K products taken in any order is within (K + 2) U sum |a b|
of the exact one.  An activation's slope is at most 1.13 (GELU's), its
float32 evaluation within 16 U of the value or of |z| (exp2, reciprocal and
erf are within a few steps each).  A result is rounded once: half a step of
its type."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
SLOPE = 1.13
TINY = 1e-37


def torch():
    import torch as _t
    return _t


def ttype(name):
    t = torch()
    return {"bf16": t.bfloat16, "f32": t.float32}[name]


def normal(seed, *shape, sigma=1.0, dtype="bf16"):
    """A device tensor of N(0, sigma) values, the same for the same seed."""
    t = torch()
    g = np.random.RandomState(seed).standard_normal(shape).astype(np.float32) * np.float32(sigma)
    return t.from_numpy(g).to(ttype(dtype)).cuda()


def strided(x, ld, fill=float("nan")):
    """A view equal to the matrix x in a buffer of ld-wide rows whose rest is `fill`."""
    t = torch()
    buf = t.full((x.shape[0], ld), fill, dtype=x.dtype, device=x.device)
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]], buf


def f64(x):
    return None if x is None else x.detach().double().cpu().numpy()


def workspace(nbytes):
    from communication_overlap_amd import ovl
    t = torch()
    ws = t.full((max(16, nbytes),), 0x7F, dtype=t.uint8, device="cuda")
    ovl.ovl_flags_reset(None, 0, ws, ws.numel())
    return ws


def sum_bound(a, b, k):
    return (k + 2) * U * (np.abs(a) @ np.abs(b))


def within(got, ref, bound, what):
    got = f64(got)
    bad = ~(np.abs(got - ref) <= bound + TINY)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(got - ref) / (bound + TINY), 0))), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off; at {i}: {got[i]} against {ref[i]}, "
                             f"bound {np.broadcast_to(bound, ref.shape)[i]}")
