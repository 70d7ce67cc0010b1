"""Helpers of the norm, scored-router and FP8 GPU tests: fp64 host copies, seeded draws, and the
rounding steps that their tolerances count."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}   # half a step, relative


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def host(t):
    """fp64 numpy copy."""
    return t.detach().cpu().double().numpy()


def codes(t):
    """fp64 values of E4M3 codes held in a uint8 tensor."""
    return host(t.cpu().view(torch.float8_e4m3fn).float())


def within(got, ref, tol, what=""):
    """|got - ref| <= tol, element by element; says the worst ratio."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    tol = np.broadcast_to(np.asarray(tol, dtype=np.float64), ref.shape)
    off = np.abs(got - ref)
    worst = float(np.max(off / np.maximum(tol, 1e-300), initial=0.0))
    print(f"  {what}: worst error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1.0, (what, worst)


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
