"""Inputs and derived error bounds for the sink-window attention and the norm + rotation."""

import math

import numpy as np
import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# Half a step of each type: the most that one rounding moves a value, relative to it.
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
# Rounding of one term of a sum kept in 32 bits; the tensor cores may drop two bits more.
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -22}


def normal(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float32).to(DT[dtype])


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def score_error(q, k, scale, dtype):
    """Bound of the error of scale * q.k (d + 2 roundings of terms whose sizes sum to at
    most |q||k|), plus the exponential's own (two steps of its argument and result)."""
    # (padding, which may hold anything, takes no part)
    q, k = (np.nan_to_num(f64(x), nan=0.0, posinf=0.0, neginf=0.0) for x in (q, k))
    size = scale * float(np.abs(q).max(initial=0) * np.abs(k).sum(-1).max(initial=0))
    return (q.shape[-1] + 4) * U[dtype] * size + 2.0 ** -20


def tol_y(y, mass, q, k, scale, dtype, keys):
    """|dy| <= sum_j |dp_j| |v_j| + one rounding: p moves by twice the scores' error (its
    exponential and the sum), by the sum's own roundings and, for bf16, by the rounding
    of the weights before the second product."""
    rel = 2 * score_error(q, k, scale, dtype) + keys * U[dtype] + (HALF[dtype] if dtype == "bf16" else 0.0)
    return rel * (1 + 2.0 ** -6) * mass + HALF[dtype] * np.abs(y) + 1e-30


def assert_within(got, ref, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - ref) - tol
    assert np.all(over <= 0), f"{what}: error {np.abs(got - ref).max():.3e}, {over.max():.3e} over its bound"


def token_major(t):
    """The same [B, H, N, d] values as a view of token-major storage."""
    return t.transpose(1, 2).contiguous().transpose(1, 2)


def fused(*ts):
    """Views of one token-major [B, N, sum of heads, d] storage."""
    buf = torch.cat([t.transpose(1, 2) for t in ts], dim=2).contiguous()
    out, h = [], 0
    for t in ts:
        out.append(buf[:, :, h:h + t.shape[1]].transpose(1, 2))
        h += t.shape[1]
    return out


def scale_of(d):
    return 1.0 / math.sqrt(d)
