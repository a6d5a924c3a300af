"""The activations of the fused products against fp64, relative to their own value, tails included.

With alpha = 0 the epilogue's argument is the bias, bit for bit. Bounds, for correctly rounded fp32 operations
(2^-24 each), exp2 within 2^-22 and reciprocals within 2^-23:

SiLU: v / (1 + e), e = 2^y, y = -v log2(e) rounded twice: e is within |v| 2^-23 + 2^-22; the sum, the pair's
reciprocal (1 / (d0 d1), times d1: 2^-24 + 2^-23 + 2^-24) and the product add 2^-21.4: below 2^-20 + |v| 2^-23.
GELU_TANH: the same of w = C v (1 + A v^2), whose five roundings move it by 2^-21.6 |w|: 2^-20 + |w| 2^-21.
Both stop at e = 2^60: below it (v < -41.5, or w) the result is between 0 and -41.5 / 2^60 > -2^-54.
GELU: -|v| Q(|v|) + max(v, 0), Q = R exp(-v^2 / 2). The exponent is rounded twice (v^2 2^-24 of Q, its constant
v^2 2^-26), exp2 2^-22; the polynomial is within 2^-23.3 of R, its eight steps add at most 2^-22.5 (the terms'
magnitudes sum to 1.8 of R), t (5 2^-24 off) moves R by at most 2.7 times as much, three products add 3 2^-24:
1.5e-6 in all, below 2^-19 + v^2 2^-23. Where exp(-v^2 / 2) is below 2^-126 it is 0, and so is the negative tail.
A stored value adds half a step of its type (tests/fused_refs.py)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_08_b200 as nv
from fused_refs import DTYPES, act, check, operand, stored
from helpers import tile_np

pytestmark = pytest.mark.gpu

C = 2 * np.sqrt(2 / np.pi)
K = 2048
PLANS = [(1, {"cluster": 1}), (1, {"cluster": 8}), (40, {"cluster": 1}), (64, {"cluster": 4}), (130, {"bn": 128, "cluster": 1}),
         (130, {"bn": 128, "cluster": 4}), (300, {"bn": 256, "cluster": 1, "pair": 2})]
RANGES = {"[-5, -3]": (-5.0, -3.0), "[-13, 13]": (-13.0, 13.0), "[-1, 1]": (-1.0, 1.0), "[-40, -5]": (-40.0, -5.0)}


def relative(z, name):
    if name == "gelu":
        return 2.0 ** -19 + z * z * 2.0 ** -23
    w = z if name == "silu" else C * z * (1 + 0.044715 * z * z)
    return 2.0 ** -20 + np.abs(w) * (2.0 ** -23 if name == "silu" else 2.0 ** -21)


@pytest.mark.parametrize("span", RANGES)
@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,plan", PLANS, ids=str)
def test_relative_error(cuda_device, M, plan, name, span):
    d, N = cuda_device, 2048
    rng = np.random.default_rng(M)
    lo, hi = RANGES[span]
    z = np.linspace(lo, hi, N).astype(np.float32)
    Aq, sa = operand(rng, M, K)
    Bq, sb = operand(rng, N, K)
    on = lambda a: torch.from_numpy(a).to(d)  # noqa: E731
    args = (on(Aq), on(tile_np(sa, K)), on(Bq), on(tile_np(sb, K)), torch.zeros(1, device=d))
    x = np.broadcast_to(z.astype(np.float64), (M, N))
    want = act(x, name)
    err = relative(x, name) * np.abs(want) + (2.0 ** -126 * 13 if name == "gelu" else 2.0 ** -54)
    for dtype in DTYPES:
        with nv.plan_override(**plan):
            out = nv.gemm_epilogue(*args, bias=on(z), act=name, out_dtype=dtype)
        check(out, want, stored(want, err, dtype), f"{name} {dtype}")


def test_half_precision_gelu_is_the_nearest_or_next_value(cuda_device):
    """fp16 and bf16 GELU of [-5, -3]: half a step of the type, and the fp32 value's (2^-19 + 25 2^-23) < 2^-17 of itself."""
    d, N = cuda_device, 4096
    z = np.linspace(-5, -3, N).astype(np.float32)
    rng = np.random.default_rng(7)
    Aq, sa = operand(rng, 2, 256)
    Bq, sb = operand(rng, N, 256)
    on = lambda a: torch.from_numpy(a).to(d)  # noqa: E731
    want = act(z.astype(np.float64), "gelu")
    for dtype in (torch.float16, torch.bfloat16):
        out = nv.gemm_epilogue(on(Aq), on(tile_np(sa, 256)), on(Bq), on(tile_np(sb, 256)), torch.zeros(1, device=d), bias=on(z),
                               act="gelu", out_dtype=dtype)[0].double().cpu().numpy()
        ulp = 2.0 ** np.maximum(np.floor(np.log2(np.abs(want))), np.log2(torch.finfo(dtype).tiny)) * torch.finfo(dtype).eps
        assert (np.abs(out - want) <= ulp / 2 + 2.0 ** -17 * np.abs(want)).all()
