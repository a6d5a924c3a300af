"""The fused calls run together as a feed-forward block: residual add + norm -> NVFP4, gated product -> NVFP4,
down projection + residual; and its gradients through frozen weights. Every stage is checked against fp64 on
the very codes that the stage before wrote, and the captured block gives the eager bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_08_b200 as nv
import oracle
from fused_refs import act, act_err, act_grad, act_grad_err, check, stored
from test_fused_products_gpu import check_quantised
from test_residual_norm_gpu import EPS, f64, norm64

pytestmark = pytest.mark.gpu


def weight(d, rows, K, seed):
    w = 0.05 * torch.randn(rows, K, device=d, generator=torch.Generator(d).manual_seed(seed))
    gs = nv.global_scale(w)
    q, sf = nv.quantize(w, gs)
    return q, sf, gs


def untile(sf, rows, K):
    r, c = np.arange(rows)[:, None], np.arange(K // 16)[None, :]
    return sf.cpu().numpy()[((r // 128) * (K // 64) + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4]


def exact_product(q, sf_tiled, wq, wsf, alpha):
    M, K = q.shape[0], 2 * q.shape[1]
    v, S, _ = oracle.gemm(q.cpu().numpy(), untile(sf_tiled, M, K), wq.cpu().numpy(), wsf.cpu().numpy(), float(alpha))
    return v, (K + 1) * 2.0 ** -24 * abs(float(alpha)) * S + 2.0 ** -24 * np.abs(v)


class Block:
    def __init__(self, d, T, H, I, name):
        self.T, self.H, self.I, self.name, self.d = T, H, I, name, d
        self.gq, self.gsf, gg = weight(d, 2 * I, H, 1)
        self.dq, self.dsf, gd = weight(d, H, I, 2)
        self.gsf_t, self.dsf_t = nv.gate_up_sf_tile(self.gsf), nv.sf_tile(self.dsf)
        self.gn, self.gh = torch.tensor([2688.0 / 12], device=d), torch.tensor([2688.0 / 20], device=d)
        self.al, self.al_d = nv.alpha(self.gn, gg), nv.alpha(self.gh, gd)
        g = torch.Generator(d).manual_seed(T)
        self.x = torch.randn(T, H, device=d, generator=g).bfloat16()
        self.y = (0.5 * torch.randn(T, H, device=d, generator=g)).bfloat16()
        self.w = 1 + 0.2 * torch.randn(H, device=d, generator=g)

    def forward(self):
        nq, nsf, r = nv.residual_norm_quantize(self.x, self.w, self.gn, self.y, eps=EPS)
        hq, hsf = nv.gemm_glu_quantize(nq, nsf, self.gq, self.gsf_t, self.al, self.gh, act=self.name, b_ready=True)
        out = nv.gemm_epilogue(hq, hsf, self.dq, self.dsf_t, self.al_d, residual=r, b_ready=True)
        return nq, nsf, r, hq, hsf, out


@pytest.mark.parametrize("T,H,I,name", [(1, 512, 256, "silu"), (37, 768, 512, "gelu"), (64, 1024, 768, "silu"),
                                        (130, 512, 512, "gelu_tanh"), (700, 1024, 1280, "silu")])
def test_block(cuda_device, T, H, I, name):
    b = Block(cuda_device, T, H, I, name)
    nq, nsf, r, hq, hsf, out = b.forward()
    want = f64(b.x) + f64(b.y)
    check(r, want, stored(want, 2.0 ** -23 * np.abs(want), torch.bfloat16), "r")
    n, e = norm64(f64(r), "rms")
    w = f64(b.w)
    check_quantised(nq.cpu().numpy(), untile(nsf, T, H), n * w, e * np.abs(w) + 2.0 ** -23 * np.abs(n * w), float(b.gn), "norm")
    v, e = exact_product(nq, nsf, b.gq, b.gsf, b.al)
    g, u, eg, eu = v[:, :I], v[:, I:], e[:, :I], e[:, I:]
    a, ea = act(g, name), act_err(g, eg, name)
    eh = ea * np.abs(u) + np.abs(a) * eu + ea * eu + 2.0 ** -23 * np.abs(a * u)
    check_quantised(hq.cpu().numpy(), untile(hsf, T, I), a * u, eh, float(b.gh), "h")
    v, e = exact_product(hq, hsf, b.dq, b.dsf, b.al_d)
    want = v + f64(r)
    check(out, want, stored(want, e + 2.0 ** -23 * (np.abs(v) + np.abs(want)), torch.bfloat16), "out")


def test_captured_block_and_two_streams(cuda_device):
    b = Block(cuda_device, 33, 1024, 512, "silu")
    eager = b.forward()[-1]
    b.forward()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = b.forward()[-1]
    g.replay()
    assert torch.equal(captured, eager)
    b.x.add_(1.0)                                    # new inputs under the same graph
    fresh = b.forward()[-1]
    g.replay()
    assert torch.equal(captured, fresh) and not torch.equal(fresh, eager)
    # two blocks in flight on two streams (no call shares state with another)
    c = Block(cuda_device, 50, 1024, 512, "gelu")
    want = c.forward()[-1]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            o1 = b.forward()[-1]
        with torch.cuda.stream(s2):
            o2 = c.forward()[-1]
    torch.cuda.synchronize()
    assert torch.equal(o1, fresh) and torch.equal(o2, want)
    st, code = nv.last_device_error()
    assert st == 0, hex(code)


@pytest.mark.parametrize("T", [16, 300])
def test_gradient_through_frozen_weights(cuda_device, T):
    """dout -> dh (product with the transposed down weights) -> dg, du -> dx (product with the transposed
    gate_up weights), gradients quantised as any activation is."""
    d, H, I = cuda_device, 512, 768
    b = Block(d, T, H, I, "silu")
    nq, nsf, r, hq, hsf, _ = b.forward()
    dq_t, dsf_t, gd = weight(d, I, H, 3)             # stands for the transposed down weights
    gq_t, gsf_t, gg = weight(d, H, 2 * I, 4)         # and the transposed gate_up weights
    dout = torch.randn(T, H, device=d, generator=torch.Generator(d).manual_seed(9)).bfloat16()
    q, sf, gs, al = nv.quantize_dynamic(dout, gs_other=gd, tiled=True)
    dh = nv.gemm(q, sf, dq_t, nv.sf_tile(dsf_t), al, tiled=True)
    dgu = nv.gemm_glu_backward(nq, nsf, b.gq, b.gsf_t, b.al, dh, b_ready=True)
    v, e = exact_product(nq, nsf, b.gq, b.gsf, b.al)
    g, u, eg, eu = v[:, :I], v[:, I:], e[:, :I], e[:, I:]
    a, ea, da, eda = act(g, "silu"), act_err(g, eg, "silu"), act_grad(g, "silu"), act_grad_err(g, eg, "silu")
    s = f64(dh)
    dg, du = s * u * da, s * a
    edg = np.abs(s) * (np.abs(u) * eda + eu * (np.abs(da) + eda)) + 2.0 ** -22 * np.abs(dg)
    edu = np.abs(s) * ea + 2.0 ** -23 * np.abs(du)
    check(dgu, np.concatenate((dg, du), 1), np.concatenate((stored(dg, edg, torch.bfloat16), stored(du, edu, torch.bfloat16)), 1), "dgu")
    q, sf, gs, al = nv.quantize_dynamic(dgu, gs_other=gg, tiled=True)
    dx = nv.gemm(q, sf, gq_t, nv.sf_tile(gsf_t), al, tiled=True)
    v, e = exact_product(q, sf, gq_t, gsf_t, al)
    check(dx, v, stored(v, e, torch.bfloat16), "dx")


def test_outputs_belong_to_the_given_stream(cuda_device):
    """A call on another stream takes no memory that the current stream has just freed (and may still use)."""
    b = Block(cuda_device, 40, 512, 512, "silu")
    nq, nsf, r, hq, hsf, _ = b.forward()
    dh = torch.ones(b.T, b.I, device=cuda_device).bfloat16()
    s = torch.cuda.Stream()
    calls = [
        lambda **kw: nv.residual_norm(b.x, b.w, b.y, **kw),
        lambda **kw: nv.residual_norm_quantize(b.x, b.w, b.gn, b.y, tiled=False, **kw),
        lambda **kw: (nv.gate_up_sf_tile(b.gsf, **kw),),
        lambda **kw: (nv.gemm_glu(nq, nsf, b.gq, b.gsf_t, b.al, **kw),),
        lambda **kw: nv.gemm_glu_quantize(nq, nsf, b.gq, b.gsf_t, b.al, b.gh, tiled=False, **kw),
        lambda **kw: (nv.gemm_glu_backward(nq, nsf, b.gq, b.gsf_t, b.al, dh, **kw),),
        lambda **kw: (nv.gemm_epilogue(hq, hsf, b.dq, b.dsf_t, b.al_d, residual=r, **kw),),
    ]
    for call in calls:
        out = call()
        want, ptrs = [o.clone() for o in out], {o.data_ptr() for o in out}
        torch.cuda.synchronize()
        del out
        out = call(stream=s)
        s.synchronize()
        assert not ptrs & {o.data_ptr() for o in out}
        assert all(torch.equal(o, w) for o, w in zip(out, want))
