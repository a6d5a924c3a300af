"""Work of the fused operators around the NVFP4 products, in plain torch and through the library.

Five paths: the residual add with the norms around a block (norm), the product with bias, activation and residual
in its epilogue (linear), the gated feed-forward product (glu) and its backward pass (glu_grad), and the three
chained as a feed-forward block (ffn). `run` computes them in elementary torch operations in fp32, or, where
`own` is set, with the calls a user of the library makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "relu2")
EPS = 1e-6
#: Global scale of the normed activations and of the gated hidden values: 2688 / the largest magnitude expected.
AMAX_NORM, AMAX_H = 32.0, 64.0


def listed():
    return [
        # one token of a decode step: the residual add and the norm before a block
        {"name": "norm_token", "op": "norm", "T": 1, "H": 6144, "kind": "rms", "dtype": "bf16", "out": "bf16", "post": False, "gate": False},
        # a ragged batch on an fp32 residual stream, layer norm with a bias and a channel gate
        {"name": "norm_layer_ragged", "op": "norm", "T": 777, "H": 2048, "kind": "layer", "dtype": "f32", "out": "bf16", "post": False, "gate": True},
        # a long prompt, norms on both sides of the block, gated
        {"name": "norm_prompt", "op": "norm", "T": 16384, "H": 6144, "kind": "rms", "dtype": "bf16", "out": "bf16", "post": True, "gate": True},
        # one token through a down projection, added to its residual
        {"name": "linear_token", "op": "linear", "M": 1, "N": 6144, "K": 2048, "act": "none", "bias": False, "residual": True, "out": "bf16"},
        # a ragged batch through an up projection with bias and GELU
        {"name": "linear_ragged", "op": "linear", "M": 500, "N": 2048, "K": 6144, "act": "gelu", "bias": True, "residual": False, "out": "f16"},
        # a prompt through a down projection, added to its residual
        {"name": "linear_prompt", "op": "linear", "M": 8192, "N": 6144, "K": 2048, "act": "none", "bias": False, "residual": True, "out": "bf16"},
        # a few sequences decoding through a gated block of the expert size
        {"name": "glu_few", "op": "glu", "M": 16, "I": 2048, "K": 6144, "act": "silu", "out": "bf16"},
        # a prompt through a wide gated block: the largest product
        {"name": "glu_prompt", "op": "glu", "M": 4096, "I": 8192, "K": 6144, "act": "silu", "out": "bf16"},
        # gradients of the gated block for a short ragged batch
        {"name": "glu_grad_ragged", "op": "glu_grad", "M": 700, "I": 2048, "K": 6144, "act": "silu", "out": "bf16"},
        # gradients of the gated block for a training batch
        {"name": "glu_grad_batch", "op": "glu_grad", "M": 8192, "I": 2048, "K": 6144, "act": "gelu_tanh", "out": "bf16"},
        # the whole feed-forward block for one token
        {"name": "ffn_token", "op": "ffn", "M": 1, "H": 6144, "I": 2048, "act": "silu"},
        # the whole feed-forward block for an odd prompt
        {"name": "ffn_prompt", "op": "ffn", "M": 2001, "H": 6144, "I": 2048, "act": "silu"},
    ]


def _log(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("norm", "linear", "glu", "glu_grad", "ffn"))
    out = rng.choice(("bf16", "f16", "f32"))
    act = rng.choice(ACTS)
    if op == "norm":
        h = _log(rng, 64, 12288, 8)
        t = _log(rng, 1, min(16384, 16384 * 6144 // h // (BYTES[out] // 2)), 1)
        return {"op": op, "T": t, "H": h, "kind": rng.choice(("rms", "layer")), "dtype": out, "out": rng.choice(("bf16", out)),
                "post": rng.random() < 0.5, "gate": rng.random() < 0.5}
    m, k = _log(rng, 1, 4096, 1), _log(rng, 256, 6144, 256)
    if op == "linear":
        return {"op": op, "M": m, "N": _log(rng, 64, 6144, 8), "K": k, "act": act, "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "out": out}
    if op == "ffn":
        return {"op": op, "M": m, "H": k, "I": _log(rng, 256, 2048, 256), "act": act}
    return {"op": op, "M": m, "I": _log(rng, 64, 4096, 32), "K": k, "act": act, "out": out}


# ------------------------------------------------------------------ inputs

def _codes(y):
    """e2m1 codes of y, to nearest with ties to the even code: the number of rounding borders below |y|, and the sign."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return c | (torch.signbit(y).to(torch.uint8) << 3)


def _quantise(x, gs):
    """x[R, K] -> (packed codes [R, K/2], e4m3 scales [R, K/16]) with the global scale gs, in fp32."""
    r, k = x.shape
    b = x.float().view(r, k // 16, 16)
    s = ((b.abs().amax(-1) / 6.0) * gs).clamp(max=448.0).to(torch.float8_e4m3fn)
    sd = s.float()
    c = _codes(b * torch.where(sd == 0, torch.zeros_like(sd), gs / sd)[..., None]).view(r, k // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), s


def _tile(sf):
    """Row-major scales [R, K/16] -> blocks of 128 rows x 4 scales (rows padded to 128 with zeros), flat."""
    r, c = sf.shape
    p = torch.zeros((r + 127) // 128 * 128, c, dtype=torch.uint8, device=sf.device)
    p[:r] = sf.view(torch.uint8)
    return p.view(-1, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _interleave(sf):
    """Gate rows then up rows -> groups of 16 gate rows and their 16 up rows."""
    r, c = sf.shape
    return sf.view(2, r // 32, 16, c).transpose(0, 1).reshape(r, c)


def _operand(g, rows, k, sigma, gated=False):
    """A random operand, quantised as a user's program keeps it: codes, tiled scales and its global scale."""
    x = torch.randn(rows, k, generator=g, device="cuda") * sigma
    gs = 2688.0 / x.abs().max()
    q, sf = _quantise(x, gs)
    sf = sf.view(torch.uint8)
    return q, _tile(_interleave(sf) if gated else sf), gs.reshape(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    s = {"case": case, "op": case["op"]}
    if case["op"] == "norm":
        t, h, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        channel = torch.exp(0.5 * rand(h))  # some channels of a residual stream are much larger than others
        s |= {"x": (rand(t, h) * channel).to(dt), "y": (rand(t, h) * 0.5).to(dt), "w": 1 + 0.1 * rand(h),
              "b": 0.1 * rand(h) if case["kind"] == "layer" else None, "post": 1 + 0.1 * rand(h) if case["post"] else None,
              "gate": 0.5 + 0.1 * rand(h) if case["gate"] else None, "scale": 0.75,
              "r": torch.empty(t, h, dtype=dt, device="cuda"), "out": torch.empty(t, h, dtype=DTYPES[case["out"]], device="cuda")}
    elif case["op"] == "linear":
        m, n, k, dt = case["M"], case["N"], case["K"], DTYPES[case["out"]]
        a, sa, ga = _operand(g, m, k, 1.0)
        b, sb, gb = _operand(g, n, k, 0.02)
        s |= {"a": a, "sa": sa, "b": b, "sb": sb, "alpha": 1.0 / (ga * gb), "bias": 0.5 * rand(n) if case["bias"] else None,
              "residual": rand(m, n).to(dt) if case["residual"] else None, "scale": 0.75, "out": torch.empty(m, n, dtype=dt, device="cuda")}
    elif case["op"] in ("glu", "glu_grad"):
        m, i, k, dt = case["M"], case["I"], case["K"], DTYPES[case["out"]]
        a, sa, ga = _operand(g, m, k, 1.0)
        b, sb, gb = _operand(g, 2 * i, k, 0.02, gated=True)
        s |= {"a": a, "sa": sa, "b": b, "sb": sb, "alpha": 1.0 / (ga * gb)}
        if case["op"] == "glu":
            s["out"] = torch.empty(m, i, dtype=dt, device="cuda")
        else:
            s |= {"dh": (0.1 * rand(m, i)).to(dt), "out": torch.empty(m, 2 * i, dtype=dt, device="cuda")}
    else:
        m, h, i = case["M"], case["H"], case["I"]
        b, sb, gb = _operand(g, 2 * i, h, 0.02, gated=True)
        d, sd, gd = _operand(g, h, i, 0.02)
        gn, gh = torch.full((1,), 2688.0 / AMAX_NORM, device="cuda"), torch.full((1,), 2688.0 / AMAX_H, device="cuda")
        u8 = lambda *z: torch.zeros(*z, dtype=torch.uint8, device="cuda")  # noqa: E731
        s |= {"x": rand(m, h).to(torch.bfloat16), "y": (0.5 * rand(m, h)).to(torch.bfloat16), "w": 1 + 0.1 * rand(h), "gn": gn, "gh": gh,
              "b": b, "sb": sb, "alpha": 1.0 / (gn * gb), "d": d, "sd": sd, "alpha_d": 1.0 / (gh * gd),
              "r": torch.empty(m, h, dtype=torch.bfloat16, device="cuda"), "out": torch.empty(m, h, dtype=torch.bfloat16, device="cuda"),
              "nq": u8(m, h // 2), "nsf": u8((m + 127) // 128 * 128 * (h // 16)),
              "hq": u8(m, i // 2), "hsf": u8((m + 127) // 128 * 128 * (i // 16))}
    return s


# ------------------------------------------------------------------ the plain forms

def _untile(sf, rows, cols):
    """The inverse of _tile."""
    return sf.view(-1, cols // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, cols)[:rows]


def _natural(sf):
    """The inverse of _interleave."""
    r, c = sf.shape
    return sf.reshape(r // 32, 2, 16, c).transpose(0, 1).reshape(r, c)


def _values(q, sf):
    """The operand that packed codes and row-major scales stand for, in fp32."""
    r, k = q.shape[0], 2 * q.shape[1]
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    v = lut[torch.stack((q & 15, q >> 4), -1).view(r, k).int()]
    return (v.view(r, k // 16, 16) * sf.view(torch.float8_e4m3fn).float()[..., None]).view(r, k)


def _product(a, sa, b, sb, alpha, gated=False):
    cols = a.shape[1] // 8
    sb = _untile(sb, b.shape[0], cols)
    return alpha * (_values(a, _untile(sa, a.shape[0], cols)) @ _values(b, _natural(sb) if gated else sb).t())


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "relu2":
        return v.clamp(min=0).square()
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _act_grad(v, act):
    if act == "relu":
        return (v > 0).float()
    if act == "relu2":
        return 2 * v.clamp(min=0)
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def _norm(z, kind):
    if kind == "layer":
        z = z - z.mean(-1, keepdim=True)
    return z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)


def _residual_norm(s, kind, scale, w, b=None, post=None, gate=None):
    v = s["y"].float()
    if post is not None:
        v = _norm(v, kind) * post
    if gate is not None:
        v = v * gate
    r = (s["x"].float() + scale * v).to(s["x"].dtype)
    n = _norm(r.float(), kind) * w
    return r, n if b is None else n + b


def _plain(s):
    c, op = s["case"], s["op"]
    if op == "norm":
        r, n = _residual_norm(s, c["kind"], s["scale"], s["w"], s["b"], s["post"], s["gate"])
        return {"r": r, "out": n.to(DTYPES[c["out"]])}
    if op == "linear":
        v = _product(s["a"], s["sa"], s["b"], s["sb"], s["alpha"])
        v = _act(v if s["bias"] is None else v + s["bias"], c["act"])
        v = v if s["residual"] is None else v + s["scale"] * s["residual"].float()
        return v.to(DTYPES[c["out"]])
    if op in ("glu", "glu_grad"):
        g, u = _product(s["a"], s["sa"], s["b"], s["sb"], s["alpha"], gated=True).chunk(2, -1)
        if op == "glu":
            return (_act(g, c["act"]) * u).to(DTYPES[c["out"]])
        dh = s["dh"].float()
        return torch.cat((dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])), -1).to(DTYPES[c["out"]])
    r, n = _residual_norm(s, "rms", 1.0, s["w"])
    q, sf = _quantise(n, s["gn"])
    g, u = _product(q, _tile(sf), s["b"], s["sb"], s["alpha"], gated=True).chunk(2, -1)
    q, sf = _quantise(_act(g, c["act"]) * u, s["gh"])
    v = _product(q, _tile(sf), s["d"], s["sd"], s["alpha_d"])
    return {"r": r, "out": (v + r.float()).to(torch.bfloat16)}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import nvfp4_block_scaled_08_b200 as nv
    c, op = s["case"], s["op"]
    if op == "norm":
        nv.residual_norm(s["x"], s["w"], s["y"], kind=c["kind"], bias=s["b"], post_weight=s["post"], gate=s["gate"],
                         residual_scale=s["scale"], eps=EPS, r_out=s["r"], out=s["out"])
        return {"r": s["r"], "out": s["out"]}
    if op == "linear":
        return nv.gemm_epilogue(s["a"], s["sa"], s["b"], s["sb"], s["alpha"], out=s["out"], bias=s["bias"], act=c["act"],
                                residual=s["residual"], residual_scale=s["scale"], b_ready=True)
    if op == "glu":
        return nv.gemm_glu(s["a"], s["sa"], s["b"], s["sb"], s["alpha"], out=s["out"], act=c["act"], b_ready=True)
    if op == "glu_grad":
        return nv.gemm_glu_backward(s["a"], s["sa"], s["b"], s["sb"], s["alpha"], s["dh"], out=s["out"], act=c["act"], b_ready=True)
    nv.residual_norm_quantize(s["x"], s["w"], s["gn"], s["y"], eps=EPS, r_out=s["r"], q=s["nq"], sf=s["nsf"])
    nv.gemm_glu_quantize(s["nq"], s["nsf"], s["b"], s["sb"], s["alpha"], s["gh"], act=c["act"], h_q=s["hq"], h_sf=s["hsf"], b_ready=True)
    nv.gemm_epilogue(s["hq"], s["hsf"], s["d"], s["sd"], s["alpha_d"], out=s["out"], residual=s["r"], b_ready=True)
    return {"r": s["r"], "out": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _exact_e4m3(byte):
    """Values of e4m3 bytes (no sign): (8 + m) 2^(e - 10), or m 2^-9 where e = 0."""
    e, m = (byte >> 3).double(), (byte & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))


def _exact_operand(q, sf, gated):
    """out[r, k] = code value x scale, each scale fetched from its place in the tiled layout."""
    rows, k = q.shape[0], 2 * q.shape[1]
    r = torch.arange(rows, device=q.device)[:, None]
    c = torch.arange(k // 16, device=q.device)[None, :]
    if gated:  # row of the interleaved order that holds the natural row r
        j = r % (rows // 2)
        r = j // 16 * 32 + j % 16 + 16 * (r // (rows // 2))
    at = ((r // 128) * (k // 64) + c // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + c % 4
    scale = _exact_e4m3(sf.long()[at])
    out = torch.empty(rows, k, dtype=torch.float64, device=q.device)
    for half in (0, 1):
        code = (q.long() >> (4 * half)) & 15
        mag = code & 7
        v = torch.where(mag < 2, mag * 0.5, (2 + (mag & 1)) * torch.exp2((mag >> 1).double() - 2))
        out[:, half::2] = torch.where(code > 7, -v, v)
    return (out.view(rows, k // 16, 16) * scale[..., None]).view(rows, k)


def _nearest(v, grid):
    """Index of the grid value nearest to v >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, v.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = v - grid[lo], grid[hi] - v
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def _exact_quantised(x, gs):
    """The values that the codes of x stand for, times gs."""
    r, k = x.shape
    b = x.view(r, k // 16, 16)
    scales = _exact_e4m3(torch.arange(127, device=x.device))
    s = scales[_nearest(b.abs().amax(-1) / 6 * gs, scales)]
    y = torch.where(s[..., None] == 0, torch.zeros_like(b), b * (gs / s)[..., None])
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    return (torch.copysign(e2m1[_nearest(y.abs(), e2m1)], y) * s[..., None]).view(r, k)


def _exact_act(v, act):
    """(act(v), act'(v)) in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.relu(v), torch.heaviside(v, torch.zeros_like(v))
    if act == "relu2":
        return torch.relu(v) ** 2, 2 * torch.relu(v)
    if act == "silu":
        p = torch.sigmoid(v)
        return v * p, p + v * p * torch.sigmoid(-v)
    if act == "gelu":
        p = torch.special.ndtr(v)
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    p, q = torch.sigmoid(k * (v + 0.044715 * v ** 3)), torch.sigmoid(-k * (v + 0.044715 * v ** 3))
    return v * p, p + v * p * q * k * (1 + 0.134145 * v * v)


def _exact_norm(z, kind):
    if kind == "layer":
        return (z - z.mean(-1, keepdim=True)) * torch.rsqrt(z.var(-1, unbiased=False, keepdim=True) + EPS)
    return z * torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op = case["op"]
    if op in ("norm", "ffn"):
        kind = case.get("kind", "rms")
        v = f["y"]
        if "post" in f:
            v = _exact_norm(v, kind) * f["post"]
        if "gate" in f:
            v = v * f["gate"]
        r = f["x"] + s.get("scale", 1.0) * v
        # the norm is of the residual as it is stored
        n = _exact_norm(r.to(s["x"].dtype).double(), kind) * f["w"] + f.get("b", 0.0)
        if op == "norm":
            return {"r": r, "out": n}
        v = f["alpha"] * (_exact_quantised(n, f["gn"]) @ _exact_operand(s["b"], s["sb"], True).t())
        h = _exact_act(v[:, :case["I"]], case["act"])[0] * v[:, case["I"]:]
        v = f["alpha_d"] * (_exact_quantised(h, f["gh"]) @ _exact_operand(s["d"], s["sd"], False).t())
        return {"r": r, "out": v + r.to(torch.bfloat16).double()}
    v = f["alpha"] * (_exact_operand(s["a"], s["sa"], False) @ _exact_operand(s["b"], s["sb"], op != "linear").t())
    if op == "linear":
        v = _exact_act(v + f["bias"] if "bias" in f else v, case["act"])[0]
        return v + s["scale"] * f["residual"] if "residual" in f else v
    g, u = v[:, :case["I"]], v[:, case["I"]:]
    a, da = _exact_act(g, case["act"])
    return a * u if op == "glu" else torch.cat((f["dh"] * u * da, f["dh"] * a), -1)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    packed = lambda rows, k: rows * k * 9 / 16  # noqa: E731  (4-bit codes and one scale byte per 16)
    if op == "norm":
        n, e = case["T"] * case["H"], BYTES[case["dtype"]]
        vectors = 1 + (case["kind"] == "layer") + case["post"] + case["gate"]
        return {"bytes": n * (3 * e + BYTES[case["out"]]) + 4 * case["H"] * vectors, "flops": n * (10 + 6 * case["post"])}
    m = case["M"]
    if op == "ffn":
        h, i = case["H"], case["I"]
        return {"bytes": packed(2 * i, h) + packed(h, i) + 8 * m * h + 4 * h, "flops": 6 * m * h * i}
    e, k = BYTES[case["out"]], case["K"]
    if op == "linear":
        n = case["N"]
        return {"bytes": packed(m + n, k) + m * n * e * (1 + case["residual"]) + 4 * n * case["bias"], "flops": 2 * m * n * k}
    i = case["I"]
    return {"bytes": packed(m + 2 * i, k) + m * i * e * (1 if op == "glu" else 3), "flops": 4 * m * i * k}
