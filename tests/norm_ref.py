"""The gradient norm and clipping in 64 bits (numpy), and the tolerances of
their fp32 and bf16 results.

Roundings: a double sum of n terms >= 0, in any order, is off by at most
(n - 1) * 2^-53 relative (each term is rounded at most n - 1 times; the
squares themselves are exact); sqrt halves that and rounds once.  A rounding
to fp32 is off by 2^-24, to bf16 by 2^-8, relative to the value.
"""
import math

import numpy as np
import torch

U53, U24, U8 = 2.0 ** -53, 2.0 ** -24, 2.0 ** -8


def as64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy().ravel()


def total64(tensors, norm_type) -> float:
    xs = [as64(t) for t in tensors]
    x = np.concatenate(xs) if xs else np.zeros(0)
    if x.size == 0:
        return 0.0
    if norm_type == 2:
        return float(math.fsum(np.square(x))) if np.isfinite(x).all() else float(np.sum(np.square(x)))
    return float("nan") if np.isnan(x).any() else float(np.max(np.abs(x)))


def total_tol(n: int) -> float:
    """Relative: the sum's roundings, and one of the reference's own."""
    return (n + 1) * U53


def norm64(total: float, norm_type) -> float:
    return math.sqrt(total) if norm_type == 2 else total


def coef64(total: float, norm_type, max_norm: float, eps: float) -> float:
    """min(1, max_norm / (norm + eps)) of the fp32 settings, not rounded."""
    d = norm64(total, norm_type) + float(np.float32(eps))
    return 1.0 if d <= max_norm else float(np.float32(max_norm)) / d


# g * coef: coef is rounded to fp32 (its double arithmetic adds 4 roundings
# of 2^-53, far below the 1% margin), the product once more; bf16 results are
# rounded a third time.  Relative to the 64-bit product.
CLIP_F32 = 2.01 * U24
CLIP_BF16 = U8 * (1 + 3 * U24) + CLIP_F32


def check_total(got: torch.Tensor, tensors, norm_type, extra_n: int = 0):
    want, g = total64(tensors, norm_type), float(got.item())
    n = sum(t.numel() for t in tensors) + extra_n
    if math.isnan(want):
        assert math.isnan(g), (g, want)
    elif math.isinf(want) or norm_type != 2:
        assert g == want, (g, want)
    else:
        assert abs(g - want) <= total_tol(n) * want, (g, want, n)


def check_norm(got: torch.Tensor, total: float, norm_type):
    want, g = norm64(total, norm_type) if total == total else float("nan"), float(got.item())
    if math.isnan(want):
        assert math.isnan(g)
    elif want >= 2.0 ** 128:     # beyond fp32: rounding to nearest gives infinity (the total holds it)
        assert g == math.inf
    else:
        # one rounding to fp32 and one of the square root; a subnormal fp32 is
        # off by half of its fixed step of 2^-149
        assert g == want or abs(g - want) <= (U24 + 2 * U53) * want + 2.0 ** -150, (g, want)
