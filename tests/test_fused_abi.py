"""CPU checks of the fused calls' refusals: the documented status, before any CUDA call."""
import pytest

import nvfp4_block_scaled_08_b200 as nv


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def call(fn, args, **kw):
    a = dict(args)
    a.update(kw)
    return fn(*a.values())


PTRS = dict(A=0x1000, sfA=0x2000, B=0x3000, sfB=0x4000, alpha=0x5000)
COMMON = [(dict(A=None), 1), (dict(sfB=None), 1), (dict(alpha=None), 1), (dict(M=-1), 1), (dict(K=-256), 1),
          (dict(act=6), 1), (dict(act=-1), 1), (dict(flags=2), 1), (dict(K=100), 2), (dict(K=0), 2), (dict(M=1 << 31), 2),
          (dict(A=0x1004), 3), (dict(sfA=0x2008), 3), (dict(B=0x3001), 3), (dict(alpha=0x5002), 3), (dict(M=0), 0)]


@pytest.mark.parametrize("bad,status", COMMON + [
    (dict(out=None), 1), (dict(N=-8), 1), (dict(dtype=3), 1), (dict(N=12), 2), (dict(N=1 << 31), 2), (dict(out=0x6008), 3),
    (dict(bias=0x7004), 3), (dict(residual=0x80000008), 3), (dict(residual=0x6010), 1), (dict(residual=0x5FF0), 1), (dict(N=0), 0)],
    ids=str)
def test_epilogue(lib, bad, status):
    args = dict(PTRS, out=0x6000, M=16, N=768, K=512, bias=0x7000, act=2, residual=0x80000000, scale=1.0, dtype=0, flags=0, s=None)
    assert call(lib.nvfp4_gemm_epilogue, args, **bad) == status


GLU = COMMON + [(dict(I=-32), 1), (dict(I=48), 2), (dict(I=1 << 30), 2), (dict(I=0), 0)]


@pytest.mark.parametrize("bad,status", GLU + [(dict(h=None), 1), (dict(dtype=3), 1), (dict(h=0x6004), 3)], ids=str)
def test_glu(lib, bad, status):
    args = dict(PTRS, h=0x6000, M=16, I=768, K=512, act=4, dtype=0, flags=0, s=None)
    assert call(lib.nvfp4_gemm_glu, args, **bad) == status


@pytest.mark.parametrize("bad,status", GLU + [
    (dict(q=None), 1), (dict(sf=None), 1), (dict(gs=None), 1), (dict(layout=2), 1), (dict(layout=7), 1), (dict(I=96), 2),
    (dict(q=0x7008), 3), (dict(sf=0x8004), 3), (dict(gs=0x6002), 3)], ids=str)
def test_glu_quantize(lib, bad, status):
    args = dict(PTRS, M=16, I=768, K=512, act=4, gs=0x6000, q=0x7000, sf=0x8000, layout=1, flags=0, s=None)
    assert call(lib.nvfp4_gemm_glu_quantize, args, **bad) == status


@pytest.mark.parametrize("bad,status", GLU + [
    (dict(dh=None), 1), (dict(dgu=None), 1), (dict(dtype=-1), 1), (dict(dh=0x6004), 3), (dict(dgu=0x70000004), 3),
    (dict(dgu=0x6000), 1), (dict(dgu=0x6000 + 16 * 768 * 2 - 16), 1), (dict(dgu=0x1000), 1)], ids=str)
def test_glu_backward(lib, bad, status):
    args = dict(PTRS, dh=0x6000, dgu=0x70000000, M=16, I=768, K=512, act=4, dtype=0, flags=0, s=None)
    assert call(lib.nvfp4_gemm_glu_backward, args, **bad) == status


def test_gate_up_sf_tile(lib):
    f = lib.nvfp4_gate_up_sf_tile
    assert f(0x1000, 0, 64, 0x2000, None) == 0
    assert f(0x1000, -16, 64, 0x2000, None) == 1
    assert f(None, 16, 64, 0x2000, None) == 1
    assert f(0x1000, 24, 64, 0x2000, None) == 2
    assert f(0x1000, 16, 48, 0x2000, None) == 2
    # 32 rows of 4 scales in, 128 out
    for sf, out in ((0x1000, 0x1000), (0x1000, 0x1070), (0x1000, 0x0E10)):
        assert f(sf, 16, 64, out, None) == 1


NORM = [(dict(x=None), 1), (dict(w=None), 1), (dict(dtype=3), 1), (dict(norm=2), 1), (dict(rows=-1), 1), (dict(H=-8), 1),
        (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(y=None), 1), (dict(y=None, post=None), 1),
        (dict(y=None, post=None, gate=None), 1), (dict(ld_x=504), 1), (dict(ld_y=0), 1), (dict(ld_r=504), 1),
        (dict(H=516, ld_x=520, ld_y=520, ld_r=520), 2), (dict(H=32832, ld_x=40000, ld_y=40000, ld_r=40000), 2), (dict(rows=1 << 31), 2),
        (dict(x=0x1004), 3), (dict(y=0x2008), 3), (dict(w=0x3004), 3), (dict(b=0x4004), 3), (dict(post=0x5004), 3), (dict(gate=0x6004), 3),
        (dict(r=0x7004), 3), (dict(r=0x1000, ld_r=520), 1), (dict(r=0x2000, ld_r=1024), 1), (dict(ld_x=516), 3), (dict(ld_y=516), 3), (dict(ld_r=516), 3), (dict(rows=0), 0), (dict(H=0), 0)]
HEAD = dict(x=0x1000, y=0x2000, dtype=0, rows=4, H=512, ld_x=512, ld_y=512, norm=0, w=0x3000, b=0x4000, post=0x5000, gate=0x6000,
            scale=1.0, eps=1e-6, r=0x7000, ld_r=512)


@pytest.mark.parametrize("bad,status", NORM + [(dict(out=None), 1), (dict(odt=3), 1), (dict(out=0x8004), 3)], ids=str)
def test_residual_norm(lib, bad, status):
    assert call(lib.nvfp4_residual_norm, dict(HEAD, out=0x8000, odt=0, s=None), **bad) == status


@pytest.mark.parametrize("bad,status", NORM + [
    (dict(q=None), 1), (dict(sf=None), 1), (dict(gs=None), 1), (dict(layout=2), 1), (dict(H=504, layout=0), 2), (dict(H=480), 2),
    (dict(q=0x9008), 3), (dict(sf=0xA004), 3), (dict(gs=0x8002), 3)], ids=str)
def test_residual_norm_quantize(lib, bad, status):
    assert call(lib.nvfp4_residual_norm_quantize, dict(HEAD, gs=0x8000, q=0x9000, sf=0xA000, layout=1, s=None), **bad) == status


# x, y, r: 4 rows of 1024 bytes; out: 4 rows of 1024 (bf16) or 2048 bytes (fp32)
@pytest.mark.parametrize("bad", [
    dict(r=0x1010), dict(r=0x0FF0), dict(r=0x2400), dict(r=0x1C00), dict(out=0x1000), dict(out=0x1FF0), dict(out=0x7010),
    dict(out=0x6010), dict(odt=2, out=0x6010), dict(out=0x2FF0),
    # every second row of one tensor: r on the other rows but for 16 bytes, and beside an x of another stride
    dict(x=0x10000, ld_x=1024, r=0x103F0, ld_r=1024), dict(x=0x10000, ld_x=1024, r=0x10410, ld_r=1024),
    dict(x=0x10000, ld_x=1024, r=0x10400, ld_r=2048), dict(r=0x10000, ld_r=1024, out=0x11810)], ids=str)
def test_residual_norm_refuses_overlap(lib, bad):
    assert call(lib.nvfp4_residual_norm, dict(HEAD, out=0x9000, odt=0, s=None), **bad) == 1


# the same without a shared byte: the call goes on to the device check (no GPU here: not a status of the arguments)
@pytest.mark.parametrize("ok", [
    dict(), dict(r=0x1000), dict(r=0x2000), dict(r=0x0), dict(x=0x10000, ld_x=1024, r=0x10400, ld_r=1024), dict(out=0x6000 - 0x800),
    dict(r=0x10000, ld_r=4096, out=0x10400), dict(x=0x10000, ld_x=1024, y=0x10400, ld_y=1024, r=0x10400, ld_r=1024), dict(out=0x8000)], ids=str)
def test_residual_norm_takes_neighbours(lib, ok):
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses of no memory: for hosts without a GPU")
    assert call(lib.nvfp4_residual_norm, dict(HEAD, out=0x9000, odt=0, s=None), **ok) not in (0, 1, 2, 3)


@pytest.mark.parametrize("q", [0x1000, 0x13F0, 0x0FF0 - 0x3E0, 0x2010, 0x7BF0])
def test_residual_norm_quantize_refuses_overlap(lib, q):
    assert call(lib.nvfp4_residual_norm_quantize, dict(HEAD, gs=0x8000, q=q, sf=0xA000, layout=1, s=None)) == 1


def test_binding_refuses_cpu_tensors():
    import torch
    z = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        nv.residual_norm(z, torch.ones(64))
    with pytest.raises(ValueError):
        nv.gemm_glu(z.byte(), z.byte(), z.byte(), z.byte(), torch.ones(1))
