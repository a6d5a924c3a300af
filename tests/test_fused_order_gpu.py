"""The fused calls directly behind the kernels that write their vectors and scalars: a gate or bias that a product
works out, a global scale, an alpha. Those kernels let the next one start early; the results have to be those of
calls with the device idle in between."""
import pytest
import torch

import nvfp4_block_scaled_08_b200 as nv
from nvfp4_block_scaled_08_b200 import workloads

pytestmark = pytest.mark.gpu


def quantised(x):
    gs = nv.global_scale(x)
    q, sf = nv.quantize(x, gs)
    return q, nv.sf_tile(sf), gs, sf


@pytest.mark.parametrize("T,H", [(1, 1024), (40, 1024), (300, 2048)])
def test_vectors_written_just_before(cuda_device, T, H):
    """gate, weight, bias and post_weight are rows of fp32 products launched just before the norm."""
    d = cuda_device
    cond = workloads.normal(4, 2048, 1.0, 11).to(d)
    mod = workloads.normal(H, 2048, 0.02, 12).to(d)
    a, sa, ga, _ = quantised(cond)
    b, sb, gb, _ = quantised(mod)
    al = nv.alpha(ga, gb)
    x, y = workloads.normal(T, H, 1.0, 13).to(d).bfloat16(), workloads.normal(T, H, 1.0, 14).to(d).bfloat16()
    gs = torch.full((1,), 300.0, device=d)

    def run(idle, scale):
        vec = torch.full((4, H), 1e9, device=d)      # what a load before the wait would see
        alpha = al * scale
        torch.cuda.synchronize()
        nv.gemm_epilogue(a, sa, b, sb, alpha, out=vec)
        if idle:
            torch.cuda.synchronize()
        kw = dict(kind="layer", bias=vec[1], post_weight=vec[2], gate=vec[3])
        out = nv.residual_norm(x, vec[0], y, **kw)
        nv.gemm_epilogue(a, sa, b, sb, alpha, out=vec)
        q = nv.residual_norm_quantize(x, vec[0], gs, y, tiled=False, **kw)
        torch.cuda.synchronize()
        return (*out, *q, vec)

    for scale in (1.0, 0.5, 2.0):
        want = run(True, scale)
        for _ in range(5):
            assert all(torch.equal(g, w) for g, w in zip(run(False, scale), want))


@pytest.mark.parametrize("b_ready", [False, True])
@pytest.mark.parametrize("M", [1, 64, 300, 2500])
def test_scalars_and_bias_written_just_before(cuda_device, M, b_ready):
    """alpha, gs_h, the bias, the residual and dh come from kernels launched just before the products that read
    them (b_ready is about the weights alone, which stay as they are)."""
    d, H, I = cuda_device, 1024, 512
    x = workloads.normal(M, H, 1.0, 21).to(d)
    w = workloads.normal(2 * I, H, 0.05, 22).to(d)
    a, sa, ga, _ = quantised(x)
    b, sb, gb, rows = quantised(w)
    sg = nv.gate_up_sf_tile(rows)
    wide = workloads.normal(2000, 4096, 3.0, 23).to(d)
    first = nv.alpha(ga, gb)

    def run(idle):
        vec = torch.full((M, 2 * I), 1e9, device=d)
        wait = torch.cuda.synchronize if idle else (lambda: None)
        torch.cuda.synchronize()
        nv.gemm_epilogue(a, sa, b, sb, first, out=vec)
        wait()
        lin = nv.gemm_epilogue(a, sa, b, sb, first, bias=vec[M - 1], act="gelu", b_ready=b_ready)
        wait()
        res = nv.gemm_epilogue(a, sa, b, sb, first, residual=lin, b_ready=b_ready)
        gs_h = nv.global_scale(wide)
        wait()
        q, sf = nv.gemm_glu_quantize(a, sa, b, sg, first, gs_h, tiled=False, b_ready=b_ready)
        al = nv.alpha(ga, gb)
        wait()
        h = nv.gemm_glu(a, sa, b, sg, al, b_ready=b_ready)
        wait()
        dgu = nv.gemm_glu_backward(a, sa, b, sg, al, h, b_ready=b_ready)
        torch.cuda.synchronize()
        return lin, res, q, sf, h, dgu

    want = run(True)
    for _ in range(5):
        assert all(torch.equal(g, w) for g, w in zip(run(False), want))


@pytest.mark.parametrize("M,dtype", [(1, torch.bfloat16), (40, torch.float32), (3000, torch.bfloat16), (3000, torch.float32)], ids=str)
def test_quantisers_behind_a_product(cuda_device, M, dtype):
    """The quantisers, and the product that quantises its activations itself, directly behind the product that
    writes their input (and another's global scale)."""
    d, K = cuda_device, 1024
    a, sa, ga, _ = quantised(workloads.normal(M, K, 1.0, 31).to(d))
    b, sb, gb, _ = quantised(workloads.normal(K, K, 0.05, 32).to(d))
    al = nv.alpha(ga, gb)

    def run(idle):
        wait = torch.cuda.synchronize if idle else (lambda: None)
        x = torch.full((M, K), 1e9, dtype=dtype, device=d)
        torch.cuda.synchronize()
        out = []
        nv.gemm_epilogue(a, sa, b, sb, al, out=x, act="silu")
        wait()
        out += nv.quantize_dynamic(x, gs_other=gb, tiled=False)
        nv.gemm_epilogue(a, sa, b, sb, al, out=x, act="relu")
        wait()
        out += nv.mx_quantize(x, tiled=False)
        if M <= 64:
            nv.gemm_epilogue(a, sa, b, sb, al, out=x, act="gelu")
            wait()
            out.append(nv.gemm_act(x, gb, b, sb))
        torch.cuda.synchronize()
        return [o for r in out for o in (r if isinstance(r, tuple) else (r,))]

    want = run(True)
    for _ in range(5):
        got = run(False)
        assert len(got) == len(want) and all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_graphs_at_once(cuda_device):
    """Two captured blocks replayed on two streams at once: no call shares memory with another."""
    d, H, I = cuda_device, 1024, 512
    jobs = []
    for seed, M in ((41, 24), (42, 300)):
        x, y = workloads.normal(M, H, 1.0, seed).to(d).bfloat16(), workloads.normal(M, H, 0.5, seed + 50).to(d).bfloat16()
        w = 1 + workloads.normal(1, H, 0.1, seed + 100)[0].to(d)
        b, _, gb, rows = quantised(workloads.normal(2 * I, H, 0.05, seed + 150).to(d))
        sg = nv.gate_up_sf_tile(rows)
        c, sc, gc, _ = quantised(workloads.normal(H, I, 0.05, seed + 200).to(d))
        gn, gh = torch.full((1,), 300.0, device=d), torch.full((1,), 200.0, device=d)
        al, al_c = nv.alpha(gn, gb), nv.alpha(gh, gc)

        def block(x=x, y=y, w=w, b=b, sg=sg, c=c, sc=sc, gn=gn, gh=gh, al=al, al_c=al_c):
            q, sf, r = nv.residual_norm_quantize(x, w, gn, y)
            h, hs = nv.gemm_glu_quantize(q, sf, b, sg, al, gh, b_ready=True)
            out = nv.gemm_epilogue(h, hs, c, sc, al_c, residual=r, b_ready=True)
            return out, nv.gemm_glu_backward(q, sf, b, sg, al, torch.ones(x.shape[0], I, device=d, dtype=torch.bfloat16))

        want = [o.clone() for o in block()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = block()
        jobs.append((g, got, want, torch.cuda.Stream(), block))      # (block holds the inputs)
    torch.cuda.synchronize()
    for _ in range(50):
        for g, _, _, s, _ in jobs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, got, want, _, _ in jobs:
        assert all(torch.equal(o, w) for o, w in zip(got, want))
    assert nv.last_device_error() == (0, 0)
