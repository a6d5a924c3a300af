"""The residual add with the norms around a block (residual_norm, residual_norm_quantize) against fp64.

Bounds. A row sum has at most 32 + 10 roundings in sequence (32 elements of a thread, two butterflies), so a sum
of squares is within 2^-18 of itself and its inverse root within 2^-19; with the multiplications around it the
RMS norm N is within 2^-18 |N|. The layer norm's mean is off by at most 2^-18 mean|z|, which moves N by that
over the deviation, once directly and once through the variance. r is checked against its own fp64 value
(half a step of its type beyond the fp32 error); the second norm is checked on the r that the kernel stored,
which is what it is defined on."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_08_b200 as nv
from fused_refs import DTYPES, check, stored
from test_fused_products_gpu import check_quantised

pytestmark = pytest.mark.gpu

EPS = 1e-5
SHAPES = [(1, 8), (3, 16), (77, 64), (1025, 128), (4099, 104), (5, 264), (1030, 520), (200, 1024), (40, 1032), (150, 2048), (149, 4096), (33, 6144),
          (300, 6144), (300, 8192), (4, 8200), (160, 12288), (2, 32768), (200, 24576)]


def norm64(z, kind):
    """N(z) and the bound of the kernel's N(z) on the same z."""
    mean = z.mean(-1, keepdims=True) if kind == "layer" else 0.0
    c = z - mean
    sd = np.sqrt((c * c).mean(-1, keepdims=True) + EPS)
    n = c / sd
    shift = 2.0 ** -18 * np.abs(z).mean(-1, keepdims=True) / sd if kind == "layer" else 0.0
    # (the shift squared, its part of the variance, counts where the row is nearly constant)
    return n, 2.0 ** -18 * np.abs(n) + shift * (1 + np.abs(n)) + shift * shift * np.abs(n)


def vec(d, H, seed, mean, dev=0.2):
    return (mean + dev * torch.randn(H, device=d, generator=torch.Generator(d).manual_seed(seed))).float()


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    def __init__(self, d, T, H, dtype, kind, y=True, post=False, gate=False, bias=False, seed=0, offset=0.0):
        g = torch.Generator(d).manual_seed(1000 * T + H + seed)
        rnd = lambda s: (torch.randn(T, H, device=d, generator=g) * s + offset)  # noqa: E731
        self.x = rnd(2.0).to(dtype)
        self.y = rnd(0.7).to(dtype) if y else None
        self.kw = dict(kind=kind, eps=EPS, bias=vec(d, H, 1, 0.1) if bias else None, post_weight=vec(d, H, 2, 1.0) if post else None,
                       gate=vec(d, H, 3, 0.5) if gate else None, residual_scale=0.75)
        self.w, self.dtype, self.kind, self.d = vec(d, H, 4, 1.0), dtype, kind, d

    def check_r(self, r):
        x, v = f64(self.x), f64(self.y)
        e = np.zeros_like(v)
        if self.kw["post_weight"] is not None:
            n, en = norm64(v, self.kind)
            p = f64(self.kw["post_weight"])
            v, e = n * p, en * np.abs(p) + 2.0 ** -23 * np.abs(n * p)
        if self.kw["gate"] is not None:
            q = f64(self.kw["gate"])
            v, e = v * q, e * np.abs(q) + 2.0 ** -23 * np.abs(v * q)
        want = x + 0.75 * v
        check(r, want, stored(want, 0.75 * e + 2.0 ** -23 * (np.abs(x) + np.abs(v)), self.dtype), "r")

    def expected(self, r):
        n, e = norm64(f64(r), self.kind)
        w = f64(self.w)
        out, e = n * w, e * np.abs(w) + 2.0 ** -23 * np.abs(n * w)
        if self.kw["bias"] is not None:
            b = f64(self.kw["bias"])
            out, e = out + b, e + 2.0 ** -23 * (np.abs(out) + np.abs(b))
        return out, e

    def run(self, out_dtype):
        T, H = self.x.shape
        full = torch.full((T + 1, H), -77.0, dtype=out_dtype, device=self.d)
        out, r = nv.residual_norm(self.x, self.w, self.y, out=full[:T], **(self.kw if self.y is not None else dict(
            self.kw, post_weight=None, gate=None)))
        assert (full[T:] == -77.0).all()
        return out, r


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_residual_norm(cuda_device, T, H, kind):
    for i, dtype in enumerate(DTYPES):
        c = Case(cuda_device, T, H, dtype, kind, post=i != 0, gate=i != 1, bias=kind == "layer")
        for out_dtype in {dtype, DTYPES[(i + 1) % 3]}:
            out, r = c.run(out_dtype)
            c.check_r(r)
            want, e = c.expected(r)
            check(out, want, stored(want, e, out_dtype), f"{kind} {dtype} -> {out_dtype}")


@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_alone(cuda_device, T, H):
    for dtype in DTYPES:
        c = Case(cuda_device, T, H, dtype, "rms", y=False, bias=True)
        out, r = c.run(dtype)
        assert r is c.x
        want, e = c.expected(r)
        check(out, want, stored(want, e, dtype), str(dtype))


@pytest.mark.parametrize("T,H", [(1, 64), (3, 16), (77, 64), (19, 48), (4099, 128), (5, 272), (1030, 576), (129, 1024), (150, 2048), (33, 6144), (300, 6144),
                                 (4, 8256), (160, 12288), (2, 32768)])
def test_quantised(cuda_device, T, H):
    d = cuda_device
    for i, dtype in enumerate(DTYPES):
        kind = ("rms", "layer")[i % 2]
        c = Case(d, T, H, dtype, kind, post=i == 1, gate=i == 2, bias=i == 1)
        gs = torch.tensor([2688.0 / 8.0], device=d)
        for tiled in ((False, True) if H % 64 == 0 else (False,)):
            q = torch.full((T + 1, H // 2), 0xA7, dtype=torch.uint8, device=d)
            rows = (T + 127) // 128 * 128 if tiled else T
            sf = torch.full((rows * (H // 16) + 16,), 0xA7, dtype=torch.uint8, device=d)
            _, _, r = nv.residual_norm_quantize(c.x, c.w, gs, c.y, q=q[:T], sf=sf, tiled=tiled, **c.kw)
            assert (q[T:] == 0xA7).all() and (sf[rows * (H // 16):] == 0xA7).all()
            c.check_r(r)
            out, r2 = c.run(torch.float32)
            assert torch.equal(r, r2)
            s = sf[:rows * (H // 16)].cpu().numpy()
            if tiled:
                ri, ci = np.arange(T)[:, None], np.arange(H // 16)[None, :]
                at = ((ri // 128) * (H // 64) + ci // 4) * 512 + (ri % 32) * 16 + ((ri // 32) % 4) * 4 + ci % 4
                pad = np.ones(s.size, bool)
                pad[at.ravel()] = False
                assert (s[pad] == 0xA7).all()
                s = s[at]
            else:
                s = s.reshape(T, H // 16)
            want, e = c.expected(r)
            check_quantised(q[:T].cpu().numpy(), s, want, e, float(gs), f"{kind} {dtype}")
            # the quantiser's own bytes for the fp32 output of the same norm
            q2, s2 = nv.quantize(out, gs)
            assert torch.equal(q[:T], q2)
            np.testing.assert_array_equal(s, s2.cpu().numpy())


def test_rows_of_a_wider_array_and_in_place(cuda_device):
    """Strided rows, and the residual written over x or over y: the same bits."""
    d = cuda_device
    for dtype in DTYPES:
        for T, H in ((7, 1032), (300, 2048)):
            c = Case(d, T, H, dtype, "rms", post=True, gate=True)
            out, r = c.run(dtype)
            wide = torch.full((T, H + 64), -5.0, dtype=dtype, device=d)
            xs, ys, rs = wide.clone(), wide.clone(), wide.clone()
            xs[:, :H], ys[:, 8:8 + H] = c.x, c.y
            o2, r2 = nv.residual_norm(xs[:, :H], c.w, ys[:, 8:8 + H], r_out=rs[:, 16:16 + H], **c.kw)
            assert torch.equal(o2, out) and torch.equal(r2, r)
            assert (rs[:, :16] == -5).all() and (rs[:, 16 + H:] == -5).all()
            x3 = c.x.clone()
            o3, _ = nv.residual_norm(x3, c.w, c.y, r_out=x3, **c.kw)
            y4 = c.y.clone()
            o4, _ = nv.residual_norm(c.x, c.w, y4, r_out=y4, **c.kw)
            assert torch.equal(o3, out) and torch.equal(x3, r) and torch.equal(o4, out) and torch.equal(y4, r)


def test_fp32_pointers_aligned_to_16_bytes_only(cuda_device):
    """Weights and fp32 rows on 16- but not 32-byte addresses give the bits of aligned ones."""
    d = cuda_device
    shift = lambda t: torch.cat([t.new_zeros(4), t.flatten()])[4:].view(t.shape)  # noqa: E731
    for dtype in DTYPES:
        c = Case(d, 33, 1024, dtype, "layer", post=True, gate=True, bias=True)
        out, r = c.run(torch.float32)
        kw = dict(c.kw, bias=shift(c.kw["bias"]), post_weight=shift(c.kw["post_weight"]), gate=shift(c.kw["gate"]))
        w = shift(c.w)
        assert w.data_ptr() % 32 == 16
        x, y = (shift(c.x), shift(c.y)) if dtype == torch.float32 else (c.x, c.y)
        o2, r2 = nv.residual_norm(x, w, y, out=shift(torch.empty_like(out)), r_out=shift(torch.empty_like(r)) if dtype == torch.float32 else None, **kw)
        assert torch.equal(o2, out) and torch.equal(r2, r)


def test_large_mean_and_constant_rows(cuda_device):
    """A layer norm of rows whose mean dwarfs their spread, and of constant and zero rows (N = 0: out = bias)."""
    d = cuda_device
    c = Case(d, 9, 2048, torch.float32, "layer", bias=True, offset=300.0)
    c.x[3], c.y[3] = 7.0, 0.0
    c.x[4], c.y[4] = 0.0, 0.0
    out, r = c.run(torch.float32)
    want, e = c.expected(r)
    check(out, want, stored(want, e, torch.float32))
    assert torch.equal(out[3], c.kw["bias"]) and torch.equal(out[4], c.kw["bias"])
    z = Case(d, 2, 64, torch.bfloat16, "rms", y=False)
    z.x[0] = 0
    assert (z.run(torch.bfloat16)[0][0] == 0).all()
    q, sf, _ = nv.residual_norm_quantize(z.x, z.w, torch.ones(1, device=d), tiled=False)
    assert ((q[0] & 0x77) == 0).all() and (sf[0] == 0).all()


def test_offsets_past_32_bits(cuda_device):
    d, T, H = cuda_device, 270_000, 8192
    assert T * H > 2 ** 31
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=d)
    y = torch.zeros(T, H, dtype=torch.bfloat16, device=d)
    c = Case(d, 50, H, torch.bfloat16, "rms", post=True, gate=True)
    x[-50:], y[-50:] = c.x, c.y
    out, r = nv.residual_norm(x, c.w, y, r_out=x, out=y.new_zeros(T, H), **c.kw)
    # (not the bits of a call of 50 rows: the threads that share a row, and with them the order of its
    # sums, go by the number of rows)
    c.check_r(x[-50:])
    want, e = c.expected(x[-50:])
    check(out[-50:], want, stored(want, e, torch.bfloat16))
    assert not out[:-50].any()
    gs = 300.0
    q, sf, _ = nv.residual_norm_quantize(x, c.w, torch.ones(1, device=d) * gs, eps=EPS)
    ri, ci = torch.arange(T - 50, T)[:, None], torch.arange(H // 16)[None, :]
    at = ((ri // 128) * (H // 64) + ci // 4) * 512 + (ri % 32) * 16 + ((ri // 32) % 4) * 4 + ci % 4
    check_quantised(q[-50:].cpu().numpy(), sf[at.to(d)].cpu().numpy(), want, e, gs, "large")


def test_bad_rows_stay_in_their_rows(cuda_device):
    d = cuda_device
    c = Case(d, 200, 512, torch.bfloat16, "rms", post=True)
    out, r = c.run(torch.bfloat16)
    c.x[7, 3], c.y[9, 0] = float("inf"), float("nan")
    out2, r2 = c.run(torch.bfloat16)
    keep = [i for i in range(200) if i not in (7, 9)]
    assert torch.equal(out[keep], out2[keep]) and torch.equal(r[keep], r2[keep])
    assert out2[9].isnan().all() and out2[7, 3].isnan()


def test_graph_and_other_stream(cuda_device):
    d = cuda_device
    c = Case(d, 64, 4096, torch.bfloat16, "rms", post=True, gate=True)
    out, r = c.run(torch.bfloat16)
    o2, r2 = torch.empty_like(out), torch.empty_like(r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nv.residual_norm(c.x, c.w, c.y, r_out=r2, out=o2, **c.kw)
    g.replay()
    assert torch.equal(o2, out) and torch.equal(r2, r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, _ = nv.residual_norm(c.x, c.w, c.y, **c.kw)
    s.synchronize()
    assert torch.equal(o3, out)


def test_refusals(cuda_device):
    d = cuda_device
    x = torch.zeros(4, 64, device=d)
    w = torch.ones(64, device=d)
    for call in (
        lambda: nv.residual_norm(x, w[:32]),
        lambda: nv.residual_norm(x, w.bfloat16()),
        lambda: nv.residual_norm(x, w, x.bfloat16()),
        lambda: nv.residual_norm(x, w, x[:3]),
        lambda: nv.residual_norm(x, w, kind="batch"),
        lambda: nv.residual_norm(x.t(), w),
        lambda: nv.residual_norm(x, w, out=torch.zeros(4, 64, dtype=torch.int32, device=d)),
        lambda: nv.residual_norm(x.double(), w),
        lambda: nv.residual_norm_quantize(x, w, torch.ones(1, device=d), q=torch.zeros(4, 31, dtype=torch.uint8, device=d)),
        lambda: nv.residual_norm_quantize(x, w, torch.ones(1)),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: nv.residual_norm(x, w, gate=w),                           # a gate without y
        lambda: nv.residual_norm(x, w, x[:1].expand(4, 64)),              # a broadcast y: row stride 0
        lambda: nv.residual_norm(x, w, eps=-1.0),
        lambda: nv.residual_norm(x[:, :12], w[:12].contiguous()),         # H % 8
        lambda: nv.residual_norm(x[:, 1:9], w[:8].contiguous()),          # a misaligned row
        lambda: nv.residual_norm_quantize(x[:, :32], w[:32].contiguous(), torch.ones(1, device=d)),  # tiled: H % 64
    ):
        with pytest.raises(nv.Nvfp4Error):
            call()
    assert nv.residual_norm(x[:0], w)[0].shape == (0, 64)
