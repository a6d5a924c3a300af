"""Plain fp64 references and derived error bounds of the fused products and norms.

Bounds. The kernels accumulate in fp32: acc is within (K + 1) 2^-24 sum|a b| of the exact sum in any order
(the alpha multiply included), called e_v below. Activations are evaluated in fp32 from an exponential within
2^-22 of an argument rounded to 2^-23, a reciprocal within 2^-22 and, for GELU, a polynomial of erfc within
1.5e-7: each of p = sigmoid, Phi is then within 2^-20 (the argument's error counts x^2 p (1 - p) <= 0.5 times
2^-23, or as little for GELU), so act(z) is within 2^-19 |z| (relu2: of 2^-22 z^2) and act'(z) within
2^-19 (1 + |z|); an error e in z moves act(z) by at most L e, L = 1.13 bounding |act'| of all but relu2
(there 2 |z| + e), and act'(z) by at most 1.2 e (relu: 0 away from the kink, and either value within e of it;
relu2: 2 e). A stored value adds half a step of its
type, `half_step(dtype) * |value|` (and half the smallest subnormal)."""
from __future__ import annotations

import numpy as np
import torch
from scipy import special

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "relu2")
DTYPES = (torch.bfloat16, torch.float16, torch.float32)


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def stored(value, err, dtype):
    """The bound of a stored value: the error before storing, half a step, half a subnormal step."""
    sub = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    return err + half_step(dtype) * (np.abs(value) + err) + sub


def act(z, name):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "relu2":
        return np.maximum(z, 0) ** 2
    if name == "gelu":
        return z * special.ndtr(z)
    if name == "gelu_tanh":
        return z * special.expit(2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * special.expit(z)
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "relu2":
        return 2 * np.maximum(z, 0)
    if name == "gelu":
        return special.ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        c = 2 * np.sqrt(2 / np.pi)
        w = c * (z + 0.044715 * z ** 3)
        return special.expit(w) + z * special.expit(w) * special.expit(-w) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        return special.expit(z) + z * special.expit(z) * special.expit(-z)
    return np.ones_like(z)


def act_err(z, e, name):
    """How far the kernel's act may be from act(z) when its argument is within e of z."""
    if name == "relu2":
        return (2 * np.abs(z) + e) * e + 2.0 ** -22 * z * z
    return 1.13 * e + (0 if name in ("none", "relu") else 2.0 ** -19) * np.abs(z)


def act_grad_err(z, e, name):
    if name == "none":
        return np.zeros_like(z)
    if name == "relu":
        return (np.abs(z) <= e).astype(np.float64)     # either side of the kink
    if name == "relu2":
        return 2 * e + 2.0 ** -22 * np.abs(z)
    return 1.2 * e + 2.0 ** -19 * (1 + np.abs(z))


def operand(rng, rows, K, lo=0x28, hi=0x40):
    """Random packed codes and e4m3 scale bytes (0.125 to 2) of a [rows, K] operand."""
    return (rng.integers(0, 256, (rows, K // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (rows, K // 16), dtype=np.uint8))


def check(got: torch.Tensor, want: np.ndarray, bound: np.ndarray, what=""):
    g = got.detach().double().cpu().numpy()
    assert g.shape == want.shape, (g.shape, want.shape)
    assert np.isfinite(g).all(), f"{what}: not finite"
    bad = np.abs(g - want) > bound
    if bad.any():
        at = [tuple(i) for i in np.argwhere(bad)[:5]]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, e.g. "
                             f"{[(i, g[i], want[i], bound[i]) for i in at]}")
