"""The products with a fused epilogue (bias, activation, residual; the gated product in 16 / 32 bits and in
NVFP4; its gradients) against fp64 references, on every tiling: few-token tiles with and without split-K,
128- and 256-wide tiles, split-K clusters, CTA pairs with half tiles. Bounds: tests/fused_refs.py."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_08_b200 as nv
import oracle
from fused_refs import (ACTS, DTYPES, act, act_err, act_grad, act_grad_err, check, half_step, operand, stored)
from helpers import tile_np

pytestmark = pytest.mark.gpu

ALPHA = np.float32(0.01)
SENTINEL = -77.0
# plan overrides (and the M range they apply to): the planner's choice, forced clusters, forced tile widths,
# CTA pairs with and without half tiles
FEW = [{}, {"cluster": 1}, {"cluster": 2}, {"cluster": 3}, {"cluster": 5}, {"cluster": 8}]
MANY = [{}, {"bn": 128, "cluster": 1}, {"bn": 128, "cluster": 3}, {"bn": 128, "cluster": 8}, {"bn": 256, "cluster": 1, "pair": 1},
        {"bn": 256, "cluster": 4}, {"bn": 256, "cluster": 1, "pair": 2}, {"bn": 256, "cluster": 1, "pair": 3},
        {"bn": 128, "cluster": 1, "pair": 2}]


def dev_of(x, d):
    return torch.from_numpy(np.ascontiguousarray(x)).to(d)


def interleaved(a):
    """Rows [gate | up] -> groups of 16 gate rows and their 16 up rows."""
    rows = a.shape[0]
    return a.reshape(2, rows // 32, 16, -1).transpose(1, 0, 2, 3).reshape(rows, -1)


class Product:
    """A random product on the device and its exact values v with the accumulator's bound e."""

    def __init__(self, d, M, N, K, seed, gated=False):
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.d, self.rng = M, N, K, d, rng
        Aq, sa = operand(rng, M, K)
        Bq, sb = operand(rng, N, K)
        self.v, S, _ = oracle.gemm(Aq, sa, Bq, sb, ALPHA)
        self.e = (K + 1) * 2.0 ** -24 * float(ALPHA) * S + 2.0 ** -24 * np.abs(self.v)
        self.args = (dev_of(Aq, d), dev_of(tile_np(sa, K), d), dev_of(Bq, d),
                     dev_of(tile_np(interleaved(sb) if gated else sb, K), d), torch.tensor([ALPHA], device=d))
        self.sb = sb


def guarded(M, N, dtype, d, pad=2):
    full = torch.full((M + pad, N), SENTINEL, dtype=dtype, device=d)
    return full, full[:M]


def finish(full, M):
    st, code = nv.last_device_error()
    assert st == 0, hex(code)
    assert (full[M:] == SENTINEL).all(), "rows behind the output were written"


def linear_case(p, dtype, name, bias, residual, plan, scale=0.75):
    d, M, N = p.d, p.M, p.N
    b = p.rng.standard_normal(N).astype(np.float32) if bias else None
    res = torch.from_numpy(p.rng.standard_normal((M, N)).astype(np.float32)).to(dtype).to(d) if residual else None
    full, out = guarded(M, N, dtype, d)
    with nv.plan_override(**plan):
        nv.gemm_epilogue(*p.args, out=out, bias=None if b is None else dev_of(b, d), act=name, residual=res,
                         residual_scale=scale)
    finish(full, M)
    z = p.v + (0 if b is None else b.astype(np.float64))
    e = p.e + 2.0 ** -23 * (np.abs(p.v) + np.abs(z))
    want, err = act(z, name), act_err(z, e, name)
    if residual:
        r = scale * res.double().cpu().numpy()
        want, err = want + r, err + 2.0 ** -23 * (np.abs(want) + np.abs(r))
    check(out, want, stored(want, err, dtype), f"{name} {dtype} {plan}")


@pytest.mark.parametrize("plan", FEW, ids=str)
@pytest.mark.parametrize("M", [1, 16, 17, 64])
def test_linear_few_tokens(cuda_device, M, plan):
    p = Product(cuda_device, M, 328, 2048, 100 + M)
    for i, dtype in enumerate(DTYPES):
        linear_case(p, dtype, ACTS[(M + i) % 6], bias=True, residual=True, plan=plan)
    linear_case(p, torch.bfloat16, "none", bias=False, residual=False, plan=plan)


@pytest.mark.parametrize("plan", MANY, ids=str)
@pytest.mark.parametrize("M,N", [(65, 776), (300, 520), (513, 264)])
def test_linear_many_tokens(cuda_device, M, N, plan):
    p = Product(cuda_device, M, N, 2048, 200 + M)
    for i, dtype in enumerate(DTYPES):
        linear_case(p, dtype, ACTS[(M + i) % 6], bias=i != 1, residual=i != 2, plan=plan)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_activations(cuda_device, name, dtype):
    for M, K in ((3, 256), (130, 512)):
        linear_case(Product(cuda_device, M, 136, K, 300 + M), dtype, name, bias=True, residual=False, plan={})


def test_linear_without_epilogue_is_the_plain_product(cuda_device):
    for M, N, K in ((1, 768, 2048), (200, 768, 2048), (700, 2048, 4096)):
        p = Product(cuda_device, M, N, K, 400 + M)
        for dtype in DTYPES:
            assert torch.equal(nv.gemm_epilogue(*p.args, out_dtype=dtype, b_ready=True),
                               nv.gemm(*p.args, tiled=True, out_dtype=dtype))


@pytest.mark.parametrize("M", [5, 64, 300])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_residual_in_place(cuda_device, M, dtype):
    """out may be the residual itself: the same bits as with a residual of its own."""
    for plan in ({}, {"cluster": 1}, {"cluster": 4}) + (({"bn": 256, "cluster": 1, "pair": 2},) if M > 64 else ()):
        p = Product(cuda_device, M, 520, 1024, 500 + M)
        res = torch.randn(M, 520, device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(M)).to(dtype)
        with nv.plan_override(**plan):
            want = nv.gemm_epilogue(*p.args, residual=res, residual_scale=0.5, act="silu", out_dtype=dtype)
            got = nv.gemm_epilogue(*p.args, out=res, residual=res, residual_scale=0.5, act="silu")
        assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)


# ------------------------------------------------------------------ gated product

def glu_parts(p):
    I = p.N // 2
    return p.v[:, :I], p.v[:, I:], p.e[:, :I], p.e[:, I:]


def glu_expected(p, name):
    g, u, eg, eu = glu_parts(p)
    a, ea = act(g, name), act_err(g, eg, name)
    h = a * u
    return h, ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2.0 ** -23 * np.abs(h)


def glu_case(p, dtype, name, plan):
    full, out = guarded(p.M, p.N // 2, dtype, p.d)
    with nv.plan_override(**plan):
        nv.gemm_glu(*p.args, out=out, act=name)
    finish(full, p.M)
    h, e = glu_expected(p, name)
    check(out, h, stored(h, e, dtype), f"glu {name} {dtype} {plan}")


def grad_case(p, dtype, name, plan):
    M, I = p.M, p.N // 2
    dh_t = torch.from_numpy(p.rng.standard_normal((M, I)).astype(np.float32)).to(dtype).to(p.d)
    full, out = guarded(M, 2 * I, dtype, p.d)
    with nv.plan_override(**plan):
        nv.gemm_glu_backward(*p.args, dh_t, out=out, act=name)
    finish(full, M)
    g, u, eg, eu = glu_parts(p)
    dh = dh_t.double().cpu().numpy()
    a, ea, da, eda = act(g, name), act_err(g, eg, name), act_grad(g, name), act_grad_err(g, eg, name)
    dg, du = dh * u * da, dh * a
    edg = np.abs(dh) * (np.abs(u) * eda + eu * (np.abs(da) + eda)) + 2.0 ** -22 * np.abs(dg)
    edu = np.abs(dh) * ea + 2.0 ** -23 * np.abs(du)
    check(out, np.concatenate((dg, du), 1),
          np.concatenate((stored(dg, edg, dtype), stored(du, edu, dtype)), 1), f"grad {name} {dtype} {plan}")


def quant_case(p, name, plan, tiled):
    """Scales and codes against the quantiser's steps on the exact h, away from rounding borders; everywhere the
    value the codes stand for lies within half a code step of h."""
    M, I = p.M, p.N // 2
    h, e = glu_expected(p, name)
    gs = np.float32(2688.0 / max(np.abs(h).max(), 1e-3))
    hq = torch.full((M + 2, I // 2), 0xA7, dtype=torch.uint8, device=p.d)
    rows = (M + 127) // 128 * 128 if tiled else M
    hsf = torch.full((rows * (I // 16) + 32,), 0xA7, dtype=torch.uint8, device=p.d)
    with nv.plan_override(**plan):
        nv.gemm_glu_quantize(*p.args, torch.tensor([gs], device=p.d), hq[:M], hsf, act=name, tiled=tiled)
    st, code = nv.last_device_error()
    assert st == 0, hex(code)
    assert (hq[M:] == 0xA7).all() and (hsf[rows * (I // 16):] == 0xA7).all()
    q, s = hq[:M].cpu().numpy(), hsf[:rows * (I // 16)].cpu().numpy()
    if tiled:
        r, c = np.arange(M)[:, None], np.arange(I // 16)[None, :]
        at = ((r // 128) * (I // 64) + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
        pad = np.ones(s.size, bool)
        pad[at.ravel()] = False
        assert (s[pad] == 0xA7).all(), "padding scales were written"
        s = s[at]
    else:
        s = s.reshape(M, I // 16)
    check_quantised(q, s, h, e, float(gs), f"{name} {plan}")


E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)])


def check_quantised(q, s, h, e, gs, what):
    """q, s: packed codes and row-major scale bytes; h, e: the exact values and the bound of the kernel's."""
    M, I = h.shape
    amax = np.abs(h).reshape(M, I // 16, 16).max(-1)
    ea = e.reshape(M, I // 16, 16).max(-1)
    # the scale byte: nearest e4m3 to amax / 6 * gs within the bound of amax (and three fp32 roundings)
    lo = np.maximum(amax - ea, 0) / 6 * gs * (1 - 2.0 ** -21)
    hi = np.minimum((amax + ea) / 6 * gs * (1 + 2.0 ** -21), 448.0)
    mid = (E4M3[1:] + E4M3[:-1]) / 2                          # borders between neighbouring scales
    assert (s < 127).all()
    assert ((s >= np.searchsorted(mid, lo, "left")) & (s <= np.searchsorted(mid, hi, "right"))).all(), f"{what}: scales"
    codes = np.empty((M, I), np.int64)
    codes[:, 0::2], codes[:, 1::2] = q & 15, q >> 4
    sd = np.repeat(E4M3[s], 16, 1)
    y = np.divide(h * gs, sd, out=np.zeros_like(h), where=sd > 0)
    ey = np.divide(e * gs, sd, out=np.zeros_like(h), where=sd > 0) + 2.0 ** -21 * np.abs(y)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    mag = codes & 7
    ok = (mag >= np.searchsorted(mid, np.maximum(np.abs(y) - ey, 0), "left")) & (mag <= np.searchsorted(mid, np.abs(y) + ey, "right"))
    assert ok.all(), f"{what}: {int((~ok).sum())} codes, e.g. {[(tuple(i), codes[tuple(i)], y[tuple(i)]) for i in np.argwhere(~ok)[:4]]}"
    sign = (codes >> 3) == (h < 0)
    assert (sign | (np.abs(h) <= e)).all(), f"{what}: signs"


@pytest.mark.parametrize("plan", FEW, ids=str)
@pytest.mark.parametrize("M,I", [(1, 96), (16, 352), (17, 64), (64, 160), (50, 32)])
def test_glu_few_tokens(cuda_device, M, I, plan):
    p = Product(cuda_device, M, 2 * I, 2048, 600 + M, gated=True)
    for i, dtype in enumerate(DTYPES):
        glu_case(p, dtype, ACTS[(M + i) % 6], plan)
        grad_case(p, dtype, ACTS[(M + i + 2) % 6], plan)
    quant_case(p, "silu", plan, tiled=I % 64 == 0)
    quant_case(p, "gelu", plan, tiled=False)


@pytest.mark.parametrize("plan", MANY, ids=str)
@pytest.mark.parametrize("M,I", [(65, 416), (300, 160), (513, 64), (257, 320)])
def test_glu_many_tokens(cuda_device, M, I, plan):
    p = Product(cuda_device, M, 2 * I, 2048, 700 + M, gated=True)
    for i, dtype in enumerate(DTYPES):
        glu_case(p, dtype, ACTS[(M + i) % 6], plan)
        grad_case(p, dtype, ACTS[(M + i + 2) % 6], plan)
    quant_case(p, "silu", plan, tiled=I % 64 == 0)
    quant_case(p, "gelu_tanh", plan, tiled=False)


@pytest.mark.parametrize("name", ACTS)
def test_glu_activations(cuda_device, name):
    for M, K in ((3, 256), (130, 512)):
        p = Product(cuda_device, M, 256, K, 800 + M, gated=True)
        for dtype in DTYPES:
            glu_case(p, dtype, name, {})
            grad_case(p, dtype, name, {})
        quant_case(p, name, {}, tiled=True)


def test_glu_planner_pairs_with_half_tiles(cuda_device):
    """A product that the planner itself runs as CTA pairs with a last wave of half tiles."""
    p = Product(cuda_device, 1024, 2 * 2560, 4096, 901, gated=True)
    glu_case(p, torch.bfloat16, "silu", {})
    grad_case(p, torch.bfloat16, "silu", {})
    quant_case(p, "silu", {}, tiled=True)
    linear_case(Product(cuda_device, 1024, 5120, 4096, 902), torch.bfloat16, "gelu", True, True, {})


def test_gradient_against_differences(cuda_device):
    """dg and du against central differences of the forward kernel itself, g and u moved by a change of alpha
    along v: d/dt sum(dh * h((1 + t) alpha)) = sum(dg * g + du * u). Step t = 2^-6: the second-order term is
    t^2 / 6 of the third derivative, here below 2^-9 of the sum of magnitudes; fp32 outputs."""
    p = Product(cuda_device, 40, 256, 512, 77, gated=True)
    dh = torch.from_numpy(p.rng.standard_normal((40, 128)).astype(np.float32)).to(cuda_device)
    t = 2.0 ** -6
    for name in ("silu", "gelu", "gelu_tanh"):
        d = nv.gemm_glu_backward(*p.args, dh, act=name).double()
        hp = nv.gemm_glu(*p.args[:4], p.args[4] * (1 + t), act=name, out_dtype=torch.float32).double()
        hm = nv.gemm_glu(*p.args[:4], p.args[4] * (1 - t), act=name, out_dtype=torch.float32).double()
        numeric = dh.double() * (hp - hm) / (2 * t)
        v = torch.from_numpy(p.v).to(cuda_device)
        formula = d * v
        formula = formula[:, :128] + formula[:, 128:]
        # third derivative of h along t: 3 g^2 u act'' + g^3 u act''' <= |g| u (3 |g| + 2 g^2) for these
        g, u = v[:, :128].abs(), v[:, 128:].abs()
        bound = dh.double().abs() * (t * t / 6 * g * u * (3 * g + 2 * g * g) * 1.2 + 2.0 ** -17 * (1 + g) * u / t)
        assert ((numeric - formula).abs() <= bound).all()


def test_gate_up_sf_tile(cuda_device):
    for I, K in ((16, 64), (96, 256), (160, 512)):
        sf = np.random.default_rng(I).integers(0, 127, (2 * I, K // 16), dtype=np.uint8)
        got = nv.gate_up_sf_tile(dev_of(sf, cuda_device))
        np.testing.assert_array_equal(got.cpu().numpy(), tile_np(interleaved(sf), K))


@pytest.mark.parametrize("scale", [1e6, 1e22, 1e30])
def test_large_arguments(cuda_device, scale):
    """Activations far outside their curved range: act(z) is 0 or z (its square for relu2, where finite), act' 0
    or 1, at any magnitude. fp32 outputs, no overflow: the up half is scaled down by its block scales."""
    d = cuda_device
    for M in (6, 140):
        p = Product(d, M, 256, 256, 61, gated=True)
        a, sa, b, sb, al = p.args
        big = al * scale
        v = torch.from_numpy(p.v).to(d) * scale
        for name in ("gelu", "gelu_tanh", "silu", "relu", "none"):
            z = v.abs() > 1e4
            assert z.float().mean() > 0.9
            want = v if name == "none" else v.clamp(min=0)
            got = nv.gemm_epilogue(a, sa, b, nv.sf_tile(dev_of(p.sb, d)), big, act=name, out_dtype=torch.float32).double()
            assert ((got - want).abs() <= 1e-5 * want.abs() + 1e-12)[z].all(), name
            if scale < 1e15:                         # g * u stays finite
                g, u, zz = v[:, :128], v[:, 128:], z[:, :128]
                h = nv.gemm_glu(a, sa, b, sb, big, act=name, out_dtype=torch.float32).double()
                want = (g if name == "none" else g.clamp(min=0)) * u
                assert ((h - want).abs() <= 2e-5 * want.abs() + 1e-5)[zz].all(), name
            dh = torch.ones(M, 128, device=d)
            grad = nv.gemm_glu_backward(a, sa, b, sb, big, dh, act=name).double()
            g, u, zz = v[:, :128], v[:, 128:], z[:, :128]
            step = torch.ones_like(g) if name == "none" else (g > 0).double()
            assert ((grad[:, :128] - u * step).abs() <= 1e-5 * u.abs())[zz].all(), name
            assert ((grad[:, 128:] - g * step).abs() <= 1e-5 * (g * step).abs() + 1e-12)[zz].all(), name


def test_offsets_past_32_bits(cuda_device):
    """Outputs of more than 2^31 elements: the last rows equal those of a product of the last rows alone."""
    d, M, N, K = cuda_device, 140_000, 16_384, 256
    assert M * N > 2 ** 31
    rng = np.random.default_rng(5)
    Aq, sa = operand(rng, M, K)
    Bq, sb = operand(rng, N, K)
    b, sbt, al = dev_of(Bq, d), dev_of(tile_np(sb, K), d), torch.tensor([ALPHA], device=d)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device=d)
    out[-300:] = 1.5
    nv.gemm_epilogue(dev_of(Aq, d), dev_of(tile_np(sa, K), d), b, sbt, al, out=out, residual=out, residual_scale=2.0)
    last = (dev_of(Aq[-300:], d), dev_of(tile_np(sa[-300:], K), d), b, sbt, al)
    want = nv.gemm_epilogue(*last, residual=torch.full((300, N), 1.5, dtype=torch.bfloat16, device=d), residual_scale=2.0)
    assert torch.equal(out[-300:], want)
    dh = out[:, :N // 2].contiguous()
    del out
    dgu = nv.gemm_glu_backward(dev_of(Aq, d), dev_of(tile_np(sa, K), d), b, sbt, al, dh)
    assert torch.equal(dgu[-300:], nv.gemm_glu_backward(*last, dh[-300:].contiguous()))


def test_deterministic_and_replayed(cuda_device):
    """The same bits twice, from another stream, and from a captured graph replayed on new inputs."""
    d = cuda_device
    p = Product(d, 48, 1024, 2048, 31, gated=True)
    first = nv.gemm_glu(*p.args)
    dh = torch.randn(48, 512, device=d).bfloat16()
    grad = nv.gemm_glu_backward(*p.args, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = nv.gemm_glu(*p.args)
    s.synchronize()
    assert torch.equal(first, other)
    out, gout = torch.empty_like(first), torch.empty_like(grad)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.gemm_glu(*p.args, out=out)
        nv.gemm_glu_backward(*p.args, dh, out=gout)
    g.replay()
    assert torch.equal(out, first) and torch.equal(gout, grad)
    dh.mul_(2)                                       # exact in bf16: the gradient doubles bit for bit
    p.args[0].copy_(p.args[0].flip(0).contiguous())  # other codes (scales stay)
    g.replay()
    assert torch.equal(out, nv.gemm_glu(*p.args)) and torch.equal(gout, nv.gemm_glu_backward(*p.args, dh))


def test_nan_scales_stay_in_their_rows(cuda_device):
    """A NaN block scale of one token reaches that token's outputs only (padding rows of A's scales too)."""
    d = cuda_device
    for M in (5, 200):
        p = Product(d, M, 256, 512, 41, gated=True)
        a, sa, b, sb, al = p.args
        clean = nv.gemm_glu(*p.args)
        bad = sa.clone()
        full = bad.view(-1, 512 // 64, 32, 4, 4)     # [row tile, block, row % 32, row / 32, scale]
        full[0, 0, 3, 0, 0] = 0x7F                   # row 3
        if M == 5:
            full[0, :, 6:, :, :] = 0x7F              # padding rows
        out = nv.gemm_glu(a, bad, b, sb, al)
        keep = [i for i in range(M) if i != 3]
        assert out[3].isnan().all() and torch.equal(out[keep], clean[keep])


def test_refusals(cuda_device):
    d = cuda_device
    p = Product(d, 8, 128, 256, 51, gated=True)
    a, sa, b, sb, al = p.args
    for call in (
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, act="tanh"),
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, bias=torch.zeros(64, device=d)),
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, bias=torch.zeros(128, device=d, dtype=torch.bfloat16)),
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, residual=torch.zeros(8, 128, device=d)),     # bf16 out
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, out=torch.zeros(9, 128, device=d)),
        lambda: nv.gemm_epilogue(a, sa, b, sb, al, out=torch.zeros(8, 128, dtype=torch.float64, device=d)),
        lambda: nv.gemm_epilogue(a, sa[:100], b, sb, al),
        lambda: nv.gemm_epilogue(a, sa, b[:, :64], sb, al),
        lambda: nv.gemm_epilogue(a.cpu(), sa, b, sb, al),
        lambda: nv.gemm_epilogue(a, sa, b, sb.cpu(), al),
        lambda: nv.gemm_glu(a, sa, b[:127], sb, al),
        lambda: nv.gemm_glu_backward(a, sa, b, sb, al, torch.zeros(8, 63, device=d)),
        lambda: nv.gemm_glu_quantize(a, sa, b, sb, al, torch.ones(1, device=d), h_q=torch.zeros(8, 33, dtype=torch.uint8, device=d)),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nv.Nvfp4Error):               # I = 48: not a multiple of 32
        nv.gemm_glu(a, sa, b[:96], sb, al)
    with pytest.raises(nv.Nvfp4Error):               # tiled scales of h need I % 64 == 0
        nv.gemm_glu_quantize(a, sa, b[:64], sb, al, torch.ones(1, device=d))
    with pytest.raises(nv.Nvfp4Error):               # 224-wide tiles: linear scales only
        with nv.plan_override(bn=224, cluster=1):
            q = Product(d, 100, 128, 256, 52, gated=True)
            nv.gemm_glu(*q.args)
    assert nv.gemm_glu(a[:0], sa, b, sb, al).shape == (0, 64)
