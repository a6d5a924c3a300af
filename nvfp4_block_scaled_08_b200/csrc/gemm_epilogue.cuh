// gemm_epilogue.cuh -- fused epilogues of the dense NVFP4 product (EPI of GemmCfg): bias,
// activation and residual (kEpiLinear); the gated product h = act(g) * u (kEpiGlu, and
// kEpiGluQuant with h requantised to NVFP4); and its gradients (kEpiGluGrad).
//
// All arithmetic is fp32 on the fp32 accumulator; each output is rounded once, to its own type.
// A gated product's weight tile holds, per 32 rows, 16 gate rows and the 16 up rows of the same
// index (GemmCfg::GLU), so that a thread (token-major tiles) or a warp (weight-major tiles) has
// both halves of every pair and of every 16-element NVFP4 block of h: nothing of [M, 2I] is
// written to memory.
#pragma once

#include "gemm_kernel.cuh"

namespace nvfp4 {

// Activations (include/nvfp4.h, nvfp4_act).
enum : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActRelu2 = 5 };

// The special function unit takes 8 cycles per warp and operation where the others take one, so
// the activations below spend it on one exponential per element and one reciprocal per two:
// 1 / d0 = d1 (1 / (d0 d1)). Arrays come in pairs (N even; a pair's NaN or infinity stays in its
// own element). 8192 x 6144 x 2048 on 256 x 256 tiles: 51.5 us without, 58 with SiLU, 68 with bias and GELU;
// with expf, a division per element and erff 82 and 105.

__device__ __forceinline__ float exp2_approx(float x)          // 2^-22 relative, subnormal results 0
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / d of two values of 1 .. 2^61
__device__ __forceinline__ f32x2 reciprocals(f32x2 d)
{
    float d0, d1, r;
    unpack2(d, d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d0 * d1));
    return mul2(pack2(r, r), pack2(d1, d0));
}

// x, and -41.5 below: there sigmoid(x) has reached its cap, and x times it must not grow with x.
// A NaN stays one.
__device__ __forceinline__ f32x2 capped(f32x2 x)
{
    float x0, x1;
    unpack2(x, x0, x1);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x0) : "f"(-41.5f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(x1) : "f"(-41.5f));
    return pack2(x0, x1);
}

// sigmoid(x) = 1 / (1 + e) of two values, and e = exp(-x), capped at 2^60, where the sigmoid is
// negligible; 1 - sigmoid is their product (the difference would lose it where it is near 0).
__device__ __forceinline__ f32x2 sigmoids(f32x2 x, f32x2& e)
{
    constexpr float kLog2e = 1.4426950408889634f;
    float y0, y1;
    unpack2(mul2(x, pack2(-kLog2e, -kLog2e)), y0, y1);
    e = pack2(exp2_approx(fminf(y0, 60.0f)), exp2_approx(fminf(y1, 60.0f)));
    return reciprocals(add2(e, pack2(1.0f, 1.0f)));
}

// gelu_tanh(x) = x sigmoid(C x (1 + A x^2)), since (1 + tanh z) / 2 = sigmoid(2 z)
constexpr float kGeluC = 1.5957691216057308f, kGeluA = 0.044715f;   // C = 2 sqrt(2 / pi)
__device__ __forceinline__ f32x2 gelu_tanh_arg(f32x2 x)
{
    return mul2(mul2(x, pack2(kGeluC, kGeluC)), fma2(mul2(x, pack2(kGeluA, kGeluA)), x, pack2(1.0f, 1.0f)));
}

// Q(z) = 1 - Phi(z), Phi the normal distribution function, of z = min(|x|, 10^4), and e =
// exp(-x^2 / 2), for two values. Q(z) = R(z) exp(-z^2 / 2), and R falls smoothly from 1/2 towards
// 1 / (z sqrt(2 pi)): with t = 1 / (1 + p z), p = 0.305, R = c1 t + ... + c8 t^8 within 9.4e-8 of R
// itself for all z <= 13.3, beyond which e is 0 (minimax of the relative error, by Lawson's
// reweighted least squares; of the p between 0.2 and 0.5 the best). So Q, and x Q in the negative tail
// of GELU, is relatively exact, (2^-19 + z^2 2^-23) with the roundings, and no 1 - erf cancels. (An
// absolute 1.5e-7 with five terms left 6e-4 of GELU(-4.2), more than half a step of fp16; 8192 x 6144 x
// 2048 with bias and GELU took 64.3 us with it, 67.6 now.)
__device__ __forceinline__ f32x2 normal_tails(f32x2 x, f32x2& z, f32x2& e)
{
    constexpr float kHalfLog2e = 0.72134752044448170f, kP = 0.305f;
    constexpr float kC[8] = {0.121639736f, 0.122466817f, 0.103420869f, 0.121021673f,
                             -0.0379768237f, 0.185716897f, -0.152988315f, 0.0366991907f};
    float x0, x1, y0, y1;
    unpack2(x, x0, x1);
    z = pack2(fminf(fabsf(x0), 1e4f), fminf(fabsf(x1), 1e4f));
    unpack2(mul2(mul2(x, x), pack2(-kHalfLog2e, -kHalfLog2e)), y0, y1);
    e = pack2(exp2_approx(y0), exp2_approx(y1));
    const f32x2 t = reciprocals(fma2(z, pack2(kP, kP), pack2(1.0f, 1.0f)));
    f32x2 q = pack2(kC[7], kC[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) q = fma2(t, q, pack2(kC[i], kC[i]));
    return mul2(mul2(q, t), e);
}

// x Phi(x) = max(x, 0) - |x| Q(|x|)
__device__ __forceinline__ f32x2 gelu_of(f32x2 x, f32x2 z, f32x2 q)
{
    float x0, x1;
    unpack2(x, x0, x1);
    return fma2(mul2(z, pack2(-1.0f, -1.0f)), q, pack2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
}

// v = act(v) for all elements (the switch is uniform, one branch per array).
template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int32_t act)
{
    static_assert(N % 2 == 0, "pairs");
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];     // keeps NaN
            break;
        case kActRelu2:
#pragma unroll
            for (int i = 0; i < N; ++i) { const float p = v[i] < 0.0f ? 0.0f : v[i]; v[i] = p * p; }
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 z, e;
                const f32x2 x = pack2(v[i], v[i + 1]), q = normal_tails(x, z, e);
                unpack2(gelu_of(x, z, q), v[i], v[i + 1]);
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 e;
                const f32x2 x = pack2(v[i], v[i + 1]);
                unpack2(mul2(capped(x), sigmoids(gelu_tanh_arg(x), e)), v[i], v[i + 1]);
            }
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 e;
                const f32x2 x = pack2(v[i], v[i + 1]);
                unpack2(mul2(capped(x), sigmoids(x, e)), v[i], v[i + 1]);
            }
            break;
        default: break;
    }
}

// v = act(v) and d = act'(v) (0 at the kink of relu and relu2).
template <int N>
__device__ __forceinline__ void act_apply_grad(float (&v)[N], float (&d)[N], int32_t act)
{
    static_assert(N % 2 == 0, "pairs");
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int i = 0; i < N; ++i) { d[i] = v[i] > 0.0f ? 1.0f : 0.0f; v[i] = v[i] < 0.0f ? 0.0f : v[i]; }
            break;
        case kActRelu2:
#pragma unroll
            for (int i = 0; i < N; ++i) { const float p = v[i] < 0.0f ? 0.0f : v[i]; d[i] = 2.0f * p; v[i] = p * p; }
            break;
        case kActGelu:
            // Phi(x) + x phi(x)
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 z, e;
                const f32x2 x = pack2(v[i], v[i + 1]), q = normal_tails(x, z, e);
                float q0, q1, z0, z1;
                unpack2(q, q0, q1);
                unpack2(z, z0, z1);
                const f32x2 cdf = pack2(v[i] < 0.0f ? q0 : 1.0f - q0, v[i + 1] < 0.0f ? q1 : 1.0f - q1);
                const f32x2 xe = mul2(pack2(copysignf(z0, v[i]), copysignf(z1, v[i + 1])), e);
                unpack2(fma2(xe, pack2(0.3989422804014327f, 0.3989422804014327f), cdf), d[i], d[i + 1]);
                unpack2(gelu_of(x, z, q), v[i], v[i + 1]);
            }
            break;
        case kActGeluTanh:
            // p + x p (1 - p) z'(x), p = sigmoid(z), z = C x (1 + A x^2); x^2 is capped where
            // p (1 - p) is already 0, so that an overflowing z' cannot make 0 * infinity
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 e;
                const f32x2 x = pack2(v[i], v[i + 1]), p = sigmoids(gelu_tanh_arg(x), e);
                const f32x2 xx = pack2(fminf(v[i] * v[i], 1e8f), fminf(v[i + 1] * v[i + 1], 1e8f));
                const f32x2 dz = fma2(xx, pack2(3.0f * kGeluA * kGeluC, 3.0f * kGeluA * kGeluC), pack2(kGeluC, kGeluC));
                const f32x2 xp = mul2(capped(x), p);
                unpack2(fma2(mul2(xp, mul2(p, e)), dz, p), d[i], d[i + 1]);
                unpack2(xp, v[i], v[i + 1]);
            }
            break;
        case kActSilu:
            // p + x p (1 - p)
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f32x2 e;
                const f32x2 x = pack2(v[i], v[i + 1]), p = sigmoids(x, e), xp = mul2(capped(x), p);
                unpack2(fma2(xp, mul2(p, e), p), d[i], d[i + 1]);
                unpack2(xp, v[i], v[i + 1]);
            }
            break;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) d[i] = 1.0f;
            break;
    }
}

// ------------------------------------------------------------------ element access

// Two 16-bit output elements of one word as fp32.
__device__ __forceinline__ float2 unpack_out16x2(uint32_t w, int32_t dt)
{
    if (dt == kOutF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The side input (residual or dh) holds out_dtype elements and may be the output itself, so it
// is read with plain loads, each element by the thread that later writes its place, or whose
// value goes into the store that does. An element as it sits in memory, and its value:
__device__ __forceinline__ uint32_t load_side_bits(const GemmArgs& a, size_t idx)
{
    if (a.out_dtype == kOutF32) return static_cast<const uint32_t*>(a.side)[idx];
    return static_cast<const uint16_t*>(a.side)[idx];
}
__device__ __forceinline__ float side_value(const GemmArgs& a, uint32_t bits)
{
    return a.out_dtype == kOutF32 ? __uint_as_float(bits) : unpack_out16x2(bits, a.out_dtype).x;
}

// N consecutive side elements from idx (idx % N == 0, N = 4 or 8).
template <int N>
__device__ __forceinline__ void load_side(const GemmArgs& a, size_t idx, float (&v)[N])
{
    if (a.out_dtype == kOutF32) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(a.side) + idx + k);
            v[k] = f.x; v[k + 1] = f.y; v[k + 2] = f.z; v[k + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.side) + idx + k);
            const float2 lo = unpack_out16x2(w.x, a.out_dtype), hi = unpack_out16x2(w.y, a.out_dtype);
            v[k] = lo.x; v[k + 1] = lo.y; v[k + 2] = hi.x; v[k + 3] = hi.y;
        }
    }
}

// Four consecutive output elements (idx % 4 == 0): one 8- or 16-byte store.
__device__ __forceinline__ void store_out4(const GemmArgs& a, size_t idx, const float (&v)[4])
{
    if (a.out_dtype == kOutF32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + idx) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + idx) =
            make_uint2(pack_out16x2(v[0], v[1], a.out_dtype), pack_out16x2(v[2], v[3], a.out_dtype));
}

// ------------------------------------------------------------------ NVFP4 output of h

// Where the scale of block `blk` (16 elements) of row `row` of h goes.
__device__ __forceinline__ uint8_t* h_sf_at(const GemmArgs& a, int64_t row, int blk)
{
    if (a.h_sf_tiled)
        return a.h_sf + ((row >> 7) * (a.inter >> 6) + (blk >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (blk & 3);
    return a.h_sf + row * (a.inter >> 4) + blk;
}

// The quantiser's scale of a block with maximum magnitude amax, and r = gs / scale (0 for a zero
// scale): fp32, round to nearest, in the order of nvfp4_quantize. One division per 16 elements.
__device__ __forceinline__ uint32_t block_scale(float amax, float gs, float& r)
{
    const uint32_t s = f32_to_e4m3(__fmul_rn(__fdiv_rn(amax, 6.0f), gs));
    const float sd = e4m3_to_f32(s);
    r = sd == 0.0f ? 0.0f : __fdiv_rn(gs, sd);
    return s;
}

// ------------------------------------------------------------------ bias, activation, residual

// v = act(alpha * acc + bias) of N consecutive output columns; bias: N floats (null: none).
template <int N>
__device__ __forceinline__ void linear_act(const float* bias, int32_t act, float alpha, float (&v)[N])
{
    const f32x2 al = pack2(alpha, alpha);
    if (bias != nullptr) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            const float4 b = *reinterpret_cast<const float4*>(bias + k);
            unpack2(fma2(al, pack2(v[k], v[k + 1]), pack2(b.x, b.y)), v[k], v[k + 1]);
            unpack2(fma2(al, pack2(v[k + 2], v[k + 3]), pack2(b.z, b.w)), v[k + 2], v[k + 3]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; k += 2) unpack2(mul2(al, pack2(v[k], v[k + 1])), v[k], v[k + 1]);
    }
    act_apply(v, act);
}

// ------------------------------------------------------------------ few tokens (weights as the MMA M operand)

// Eight tokens' values h[] of index j, quantised: the 16 lanes of a half-warp hold the 16 indices of
// one block of each token. A reduce-scatter leaves lane i the maximum of token i % 8, so that each
// scale is worked out once (its inverse goes back to the other lanes), and a transpose of 8 x 8
// codes among 8 lanes leaves lane i eight neighbouring codes of token i % 8: 8 + 8 + 3 exchanges
// and one pair of divisions for 128 values. m, ok: this lane's token i % 8 and whether it exists.
__device__ __forceinline__ void quantise_tokens8(const GemmArgs& a, float gs, int j, const float (&h)[8], int m, bool ok)
{
    const int lane = threadIdx.x & 31;
    float v[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = fabsf(h[t]);
#pragma unroll
    for (int w = 4; w >= 1; w >>= 1) {
        const bool hi = (lane & w) != 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t >= w) break;
            const float recv = __shfl_xor_sync(0xffffffffu, hi ? v[t] : v[t + w], w);
            v[t] = fmaxf(hi ? v[t + w] : v[t], recv);
        }
    }
    float rcp;
    const uint32_t sf = block_scale(fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 8)), gs, rcp);
    uint32_t w = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const float r = __shfl_sync(0xffffffffu, rcp, (lane & 24) | t);
        w |= (f32x2_to_e2m1x2(__fmul_rn(h[t], r), 0.0f) & 0xFu) << (4 * t);
    }
    constexpr uint32_t kMask[3] = {0x0000FFFFu, 0x00FF00FFu, 0x0F0F0F0Fu};
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        const int d = 4 >> s, sh = 16 >> s;
        const uint32_t r = __shfl_xor_sync(0xffffffffu, w, d);
        w = (lane & d) ? (w & ~kMask[s]) | (r >> sh & kMask[s]) : (w & kMask[s]) | (r & kMask[s]) << sh;
    }
    if (ok) {
        // index of this lane's 8 codes: the lower or upper half of the block
        const int j8 = (j & ~15) + (lane & 8);
        *reinterpret_cast<uint32_t*>(a.h_q + static_cast<int64_t>(m) * (a.inter >> 1) + (j8 >> 1)) = w;
        if ((lane & 8) == 0) *h_sf_at(a, m, j >> 4) = static_cast<uint8_t>(sf);
    }
}

// One token's value h of index j, quantised: a half-warp holds the block. 4 + 3 exchanges.
__device__ __forceinline__ void quantise_token(const GemmArgs& a, float gs, int j, float h, int m, bool ok)
{
    float amax = fabsf(h), rcp;
#pragma unroll
    for (int w = 8; w >= 1; w >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, w));
    const uint32_t sf = block_scale(amax, gs, rcp);
    uint32_t w = (f32x2_to_e2m1x2(__fmul_rn(h, rcp), 0.0f) & 0xFu) << (4 * (j & 7));
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1) w |= __shfl_xor_sync(0xffffffffu, w, d);
    if (ok && (j & 7) == 0) {
        *reinterpret_cast<uint32_t*>(a.h_q + static_cast<int64_t>(m) * (a.inter >> 1) + (j >> 1)) = w;
        if ((j & 15) == 0) *h_sf_at(a, m, j >> 4) = static_cast<uint8_t>(sf);
    }
}

// (g, u) pairs of h index j of the N tokens m[] that exist (ok[]), with their dh (kEpiGluGrad).
template <class Cfg, int N>
__device__ __forceinline__ void glu_lane(const GemmArgs& a, float gs, const int (&m)[N], int j, float (&g)[N], const float (&u)[N],
                                         const bool (&ok)[N], const float (&dh)[N])
{
    if constexpr (Cfg::EPI == kEpiGluGrad) {
        float d[N];
        act_apply_grad(g, d, a.act_fn);
#pragma unroll
        for (int t = 0; t < N; ++t) {
            if (!ok[t]) continue;
            const size_t idx = static_cast<size_t>(m[t]) * a.N + j;
            store_out1(a, idx, dh[t] * u[t] * d[t]);
            store_out1(a, idx + a.inter, dh[t] * g[t]);
        }
    } else {
        act_apply(g, a.act_fn);
#pragma unroll
        for (int t = 0; t < N; ++t) g[t] *= u[t];
        if constexpr (Cfg::EPI == kEpiGluQuant) {
            if constexpr (N == 2) {                  // one token (the second is padding)
                quantise_token(a, gs, j, g[0], m[0], ok[0]);
            } else {
                static_assert(N == 8, "eight consecutive tokens");
                const int t = threadIdx.x & 7;
                quantise_tokens8(a, gs, j, g, m[0] + t, ok[0] && m[0] + t < a.M);
            }
        } else {
#pragma unroll
            for (int t = 0; t < N; ++t)
                if (ok[t]) store_out1(a, static_cast<size_t>(m[t]) * a.inter + j, g[t]);
        }
    }
}

// A warp's part of a swap tile without split-K: 32 weight rows (lane = row) x at most 32 tokens,
// taken in 16s. Linear: lane = output column n. Gated: lanes 0-15 hold 16 gate rows and lanes
// 16-31 their up rows; one exchange gives lane i (i < 16) both halves of tokens c .. c + 7 and
// lane 16 + i those of tokens c + 8 .. c + 15. The residual or dh elements are requested before
// the accumulator is awaited.
template <class Cfg>
struct EpiToks {
    static constexpr bool LINEAR = Cfg::EPI == kEpiLinear;
    static constexpr bool GRAD = Cfg::EPI == kEpiGluGrad;
    static constexpr int NT = Cfg::BN == 64 ? 32 : 16;          // tokens per warp
    const GemmArgs& a;
    const int quad, lane;
    uint32_t side[LINEAR ? NT : GRAD ? NT / 2 : 1];
    float bias = 0.0f;
    float gs = 0.0f;             // kEpiGluQuant: gs_h, asked for before the accumulator is awaited

    __device__ __forceinline__ EpiToks(const GemmArgs& args, int q, int l) : a(args), quad(q), lane(l) {}

    // token of element i of this lane's list, in 16-token group h that starts at column c
    __device__ __forceinline__ int token(const Tile& ti, int c, int i) const
    {
        return ti.q0 + c + (LINEAR ? i : i + (lane >= 16 ? 8 : 0));
    }

    __device__ __forceinline__ void begin(const Tile& ti, int half)
    {
        const int c_lo = half ? (Cfg::BN == 16 ? 16 : Cfg::BN / 2) : 0;
        if (c_lo >= Cfg::BN) return;
        if constexpr (Cfg::EPI == kEpiGluQuant) gs = ld_written(a.gs_h);
        if constexpr (LINEAR) {
            const int n = ti.p0 + 32 * quad + lane;
            if (a.bias != nullptr && n < a.N) bias = ld_written(a.bias + n);
            if (a.side != nullptr) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int m = token(ti, c_lo, i);
                    side[i] = m < a.M && n < a.N ? load_side_bits(a, static_cast<size_t>(m) * a.N + n) : 0u;
                }
            }
        } else if constexpr (GRAD) {
            const int j = (ti.p0 >> 1) + 16 * quad + (lane & 15);
#pragma unroll
            for (int i = 0; i < NT / 2; ++i) {
                const int m = token(ti, c_lo + 16 * (i >> 3), i & 7);
                side[i] = m < a.M && j < a.inter ? load_side_bits(a, static_cast<size_t>(m) * a.inter + j) : 0u;
            }
        }
    }

    // Tokens c .. c + 15, the h-th sixteen of the warp (h is 0 or 1, known at compile time).
    __device__ __forceinline__ void run(const Tile& ti, int h, int c, const uint32_t (&r)[16], float alpha)
    {
        if constexpr (LINEAR) {
            const int n = ti.p0 + 32 * quad + lane;
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = fmaf(alpha, __uint_as_float(r[j]), bias);
            act_apply(v, a.act_fn);
            if (a.side != nullptr) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = fmaf(a.side_scale, side_value(a, side[(NT == 32 ? 16 * h : 0) + j]), v[j]);
            }
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(v[j]);
            if (a.out_dtype != kOutF32) store_tok16<Cfg>(a, ti, quad, lane, c, o, 1.0f);
            else store_out16<Cfg>(a, ti, n, c, o, 1.0f);
        } else {
            const int j0 = (ti.p0 >> 1) + 16 * quad;
            if (j0 >= a.inter) return;               // warp-uniform
            const bool up = lane >= 16;
            int m[8];
            float g[8], u[8];
            bool ok[8];
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float lo = alpha * __uint_as_float(r[i]);        // token c + i
                const float hi = alpha * __uint_as_float(r[i + 8]);    // token c + 8 + i
                const float other = __shfl_xor_sync(0xffffffffu, up ? lo : hi, 16);
                m[i] = token(ti, c, i);
                ok[i] = m[i] < a.M;
                g[i] = up ? other : lo;
                u[i] = up ? hi : other;
                s[i] = GRAD ? side_value(a, side[GRAD ? (NT == 32 ? 8 * h : 0) + i : 0]) : 0.0f;
            }
            glu_lane<Cfg>(a, gs, m, j0 + (lane & 15), g, u, ok, s);
        }
    }
};

// ------------------------------------------------------------------ split-K

// The split-K epilogue, by both epilogue warpgroups (256 threads; row: this thread's accumulator
// row, half: its warpgroup). As in split_k_epilogue, the CTAs of a cluster hold consecutive K
// slices of one tile, every slice's accumulator goes to the ranks that own its parts by st.async,
// and each owner sums its parts over the ranks in order: deterministic. A part (chunk) is 8
// accumulator rows; where a gated product's weights are those rows, one group of 16 gate and 16 up
// rows for half of the tokens, so that every pair and block of h has one owner (8 such chunks of
// 32 rows over at most 8 ranks). begin(), before the accumulator is awaited, works out where
// everything goes (divisions by the cluster size) and requests gs_h (at its use it cost
// 0.2 of 7 us) and the first residual or dh elements.
template <class Cfg>
struct EpiSplit {
    static constexpr int BN = Cfg::BN;
    static constexpr bool LINEAR = Cfg::EPI == kEpiLinear;
    static constexpr bool GROUPS = Cfg::GLU && Cfg::SWAP;
    static constexpr int CR = GROUPS ? 32 : 8;       // rows of a chunk
    static constexpr int CW = GROUPS ? BN / 2 : BN;  // columns of a chunk
    static constexpr int CHUNKS = GROUPS ? 8 : 16;
    static constexpr int PS = CW + 4;
    static constexpr bool QUANT = Cfg::EPI == kEpiGluQuant;
    // tokens of a grouped item: c and c + CW / 2, or, quantised, eight neighbours; one where that
    // already makes at most an item per thread (BN = 16)
    static constexpr int NT = !GROUPS || BN == 16 ? 1 : QUANT ? 8 : 2;
    static constexpr int TS = QUANT ? 1 : CW / 2;
    static_assert(!QUANT || (GROUPS ? 16 * (CW / NT) : CR * (BN / 8)) % 32 == 0, "a chunk's items fill whole warps");
    static constexpr bool SIDE = LINEAR || Cfg::EPI == kEpiGluGrad;
    static constexpr int SV = LINEAR ? 8 : GROUPS ? NT : 4;      // side elements of an item
    struct Item { int m, j, src; bool ok; };         // token (row of the output), first column, offset of source 0

    const GemmArgs& a;
    const AbortState& ab;
    uint64_t* const rx_bar;
    const uint32_t rx;                               // the receive buffer (shared-memory address)
    const int row, half, tid, cs;
    // this row's (GROUPS: and token half's) place in its owner's receive buffer: a shared::cluster
    // address and the owner's barrier, or here (dst 0)
    uint32_t mine[GROUPS ? 2 : 1], dst[GROUPS ? 2 : 1], bar[GROUPS ? 2 : 1];
    int k0, n, items;                                // this rank's chunks [k0, k0 + n) and their items
    Item item0;
    float side0[SV];
    float gs = 0.0f;                                 // QUANT: gs_h, asked for in begin()

    __device__ __forceinline__ EpiSplit(const GemmArgs& args, uint8_t* smem, uint64_t* rxb, int r, int h,
                                        const AbortState& abort)
        : a(args), ab(abort), rx_bar(rxb), rx(smem_u32(smem + (Cfg::RX_OWN ? Cfg::OFF_RX : Cfg::OFF_P))),
          row(r), half(h), tid(128 * h + r), cs(args.cluster_size)
    {
    }

    __device__ __forceinline__ int first(int r) const { return (r * CHUNKS + cs - 1) / cs; }

    __device__ __forceinline__ void begin(const Tile& ti)
    {
        const int rank = static_cast<int>(cluster_ctarank());
        k0 = first(rank);
        n = first(rank + 1) - k0;
        items = GROUPS ? n * 16 * (CW / NT) : Cfg::SWAP ? n * BN : n * CR * (BN / 8);
#pragma unroll
        for (int p = 0; p < (GROUPS ? 2 : 1); ++p) {
            const int chunk = GROUPS ? 2 * (row >> 5) + p : row >> 3;
            const int owner = chunk * cs / CHUNKS;
            const int o0 = first(owner), on = first(owner + 1) - o0;
            mine[p] = rx + 4 * ((rank * on + chunk - o0) * CR + (row & (CR - 1))) * PS;
            dst[p] = owner == rank ? 0u : mapa_shared(mine[p], static_cast<uint32_t>(owner));
            bar[p] = owner == rank ? 0u : mapa_shared(smem_u32(rx_bar), static_cast<uint32_t>(owner));
        }
        if constexpr (QUANT) gs = ld_written(a.gs_h);
        if constexpr (SIDE) item0 = item_of(ti, tid);
        if constexpr (SIDE) {
            if (a.side != nullptr && tid < items) load_item_side(item0, side0);
        }
    }

    __device__ __forceinline__ Item item_of(const Tile& ti, int item) const
    {
        Item it;
        if constexpr (GROUPS) {
            // (index of the group, token, chunk): a half-warp holds one block of one token
            const int i = item & 15, k = (item >> 4) / (CW / NT);
            const int c = (item >> 4) % (CW / NT) * (QUANT ? NT : 1);
            const int chunk = k0 + k;
            it.m = ti.q0 + (chunk & 1) * CW + c;
            it.j = (ti.p0 >> 1) + 16 * (chunk >> 1) + i;
            it.src = (k * CR + i) * PS + c;
            it.ok = it.m < a.M && it.j < a.inter;
        } else if constexpr (Cfg::SWAP) {
            // (chunk, token): eight output columns, neighbouring chunks by neighbouring threads
            const int c = item / n, k = item - c * n;
            it.m = ti.q0 + c;
            it.j = ti.p0 + 8 * (k0 + k);
            it.src = k * CR * PS + c;
            it.ok = it.m < a.M && it.j < a.N;
        } else {
            // (column group, chunk row): eight output columns, or four indices of h
            const int g = item % (BN / 8), r = item / (BN / 8);
            it.m = ti.p0 + 8 * k0 + r;
            if constexpr (LINEAR) {
                it.j = ti.q0 + 8 * g;
                it.src = r * PS + 8 * g;
                it.ok = it.m < a.M && it.j < a.N;
            } else {
                it.j = ((ti.q0 + 32 * (g >> 2)) >> 1) + 4 * (g & 3);
                it.src = r * PS + 32 * (g >> 2) + 4 * (g & 3);
                it.ok = it.m < a.M && it.j < a.inter;
            }
        }
        return it;
    }

    __device__ __forceinline__ void load_item_side(const Item& it, float (&s)[SV]) const
    {
        const int64_t ld = LINEAR ? a.N : a.inter;
        if constexpr (GROUPS) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                s[t] = it.j < a.inter && it.m + t * TS < a.M
                           ? side_value(a, load_side_bits(a, (it.m + t * TS) * ld + it.j)) : 0.0f;
        } else {
            if (it.ok) load_side(a, it.m * ld + it.j, s);
        }
    }

    __device__ __forceinline__ void finish(const Tile& ti, uint32_t tacc, float alpha)
    {
        if (!Cfg::RX_OWN && cs > 1) { cluster_arrive(); cluster_wait(); }

        // 1. this warpgroup's columns of its row to their owners
        {
            constexpr int SPAN = BN == 16 ? 16 : BN / 2;             // (16 columns: all by the first)
            const int c_end = half * SPAN + SPAN < BN ? half * SPAN + SPAN : BN;
            for (int c = half * SPAN; c < c_end; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(tacc + c, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // GROUPS: the token half of these four columns
                    const int p = !GROUPS ? 0 : BN == 16 ? i >> 1 : half;
                    const int cc = GROUPS ? (c + 4 * i) & (CW - 1) : c + 4 * i;
                    const float4 f = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                 __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                    const uint32_t d = GROUPS && p ? dst[GROUPS ? 1 : 0] : dst[0];
                    if (d == 0u) sts_f4((GROUPS && p ? mine[GROUPS ? 1 : 0] : mine[0]) + 4 * cc, f);
                    else st_async_f4(d + 4 * cc, f.x, f.y, f.z, f.w, GROUPS && p ? bar[GROUPS ? 1 : 0] : bar[0]);
                }
            }
        }

        // 2. wait (bounded) for the other ranks' parts; the barrier publishes this CTA's own
        bool ok = true;
        if (cs > 1) {
            if (tid == 0) mbar_arrive_expect_tx(rx_bar, static_cast<uint32_t>((cs - 1) * n * CR * CW * 4));
            ok = mbar_wait(rx_bar, 0, ab, kErrSplitRx);
        }
        __syncwarp();
        ok = named_bar_and(2, 256, ok);
        if (!ok) return;

        // 3. sum over the ranks in order and finish. (QUANT: lanes exchange values, in whole warps of
        // items.)
        const int step = n * CR * PS;                    // from one rank's copy to the next
        for (int item = tid; item < items; item += 256) {
            const Item it = SIDE && item == tid ? item0 : item_of(ti, item);
            float s[SV];
            if constexpr (SIDE) {
                if (item == tid) {
#pragma unroll
                    for (int i = 0; i < SV; ++i) s[i] = side0[i];
                } else if (a.side != nullptr) {
                    load_item_side(it, s);
                }
            }
            if constexpr (LINEAR) {
                if (!it.ok) continue;
                float v[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] = 0.0f;
                for (int q = 0; q < cs; ++q) {
                    const uint32_t p = rx + 4 * (q * step + it.src);
                    if constexpr (Cfg::SWAP) {
#pragma unroll
                        for (int t = 0; t < 8; ++t) v[t] += lds_f32(p + 4 * t * PS);
                    } else {
#pragma unroll
                        for (int t = 0; t < 8; t += 4) {
                            const float4 x = lds_f4(p + 4 * t);
                            v[t] += x.x; v[t + 1] += x.y; v[t + 2] += x.z; v[t + 3] += x.w;
                        }
                    }
                }
                linear_act(a.bias != nullptr ? a.bias + it.j : nullptr, a.act_fn, alpha, v);
                if (a.side != nullptr) {
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[t] = fmaf(a.side_scale, s[t], v[t]);
                }
                store_out8(a, static_cast<size_t>(it.m) * a.N + it.j, v);
            } else if constexpr (GROUPS) {
                constexpr int NA = NT == 1 ? 2 : NT;                 // (the activations take pairs)
                float g[NA], u[NA], dh[NA];
                int m[NA];
                bool here[NA];
#pragma unroll
                for (int t = 0; t < NA; ++t) g[t] = u[t] = 0.0f;
                for (int q = 0; q < cs; ++q) {
                    const uint32_t p = rx + 4 * (q * step + it.src);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        g[t] += lds_f32(p + 4 * t * TS);
                        u[t] += lds_f32(p + 4 * (16 * PS + t * TS));
                    }
                }
#pragma unroll
                for (int t = 0; t < NA; ++t) {
                    g[t] *= alpha;
                    u[t] *= alpha;
                    m[t] = it.m + t * TS;
                    here[t] = t < NT && m[t] < a.M && it.j < a.inter;
                    dh[t] = SIDE && t < NT ? s[t < SV ? t : 0] : 0.0f;
                }
                glu_lane<Cfg>(a, gs, m, it.j, g, u, here, dh);
            } else {
                float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int q = 0; q < cs; ++q) {
                    const uint32_t p = rx + 4 * (q * step + it.src);
                    const float4 x = lds_f4(p), y = lds_f4(p + 64);
                    g[0] += x.x; g[1] += x.y; g[2] += x.z; g[3] += x.w;
                    u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) { g[i] *= alpha; u[i] *= alpha; }
                if constexpr (Cfg::EPI == kEpiGluGrad) {
                    if (!it.ok) continue;                // no exchange below
                    float d[4];
                    act_apply_grad(g, d, a.act_fn);
#pragma unroll
                    for (int i = 0; i < 4; ++i) { d[i] = s[i] * u[i] * d[i]; g[i] = s[i] * g[i]; }
                    const size_t idx = static_cast<size_t>(it.m) * a.N + it.j;
                    store_out4(a, idx, d);
                    store_out4(a, idx + a.inter, g);
                } else {
                    act_apply(g, a.act_fn);
#pragma unroll
                    for (int i = 0; i < 4; ++i) g[i] *= u[i];
                    if constexpr (Cfg::EPI == kEpiGlu) {
                        if (it.ok) store_out4(a, static_cast<size_t>(it.m) * a.inter + it.j, g);
                    } else {
                        // the four lanes of a block are neighbours
                        float amax = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3]))), rcp;
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                        const uint32_t sf = block_scale(amax, gs, rcp);
                        const uint32_t q = f32x2_to_e2m1x2(__fmul_rn(g[0], rcp), __fmul_rn(g[1], rcp)) |
                                           f32x2_to_e2m1x2(__fmul_rn(g[2], rcp), __fmul_rn(g[3], rcp)) << 8;
                        if (it.ok) {
                            *reinterpret_cast<uint16_t*>(a.h_q + static_cast<int64_t>(it.m) * (a.inter >> 1) + (it.j >> 1)) =
                                static_cast<uint16_t>(q);
                            if ((it.j & 15) == 0) *h_sf_at(a, it.m, it.j >> 4) = static_cast<uint8_t>(sf);
                        }
                    }
                }
            }
        }
    }
};

// ------------------------------------------------------------------ token-major tiles

// A warp's part of a token-major tile: 32 token rows (lane = row) x up to two chunks of 64
// accumulator columns, taken in pieces of 32. No lane exchanges data with another: results go from
// registers to memory, 32 or 64 bytes of a row per lane in whole sectors; the residual or dh comes
// in as boxes of 64 bytes x 32 rows by TMA into two buffers per warp (64-byte swizzle: a lane's
// four 16-byte pieces of its row are conflict-free), the first two requested before the accumulator
// is awaited, each next one as soon as its buffer has been read. 8192 x 6144 x 2048 without and with a
// residual, and in fp32: 51.3, 64.5 and 105 us. (Results as boxes by TMA through the same buffers,
// where a load waits for the store before it: 52.6, 66 and 111; the next tile's first boxes
// requested a tile ahead: no faster.) The residual's own cost there is one of power: 90 thousand cycles
// at 1.54 GHz against 87 at 1.75.
//
// The loops over chunks and pieces are not unrolled: the epilogue's straight-line code would
// otherwise pass the instruction cache once per tile and warp (without activation 68 us unrolled,
// with transposes among the lanes for the stores).
//
// Per 32-column piece: kEpiLinear one box of a 16-bit type or two of fp32; the gated ones 16
// indices of h ([16 gate, 16 up] columns): half a box of a 16-bit type or one of fp32.
template <class Cfg>
struct EpiRows {
    static constexpr bool LINEAR = Cfg::EPI == kEpiLinear;
    static constexpr bool GRAD = Cfg::EPI == kEpiGluGrad;
    static constexpr bool QUANT = Cfg::EPI == kEpiGluQuant;
    static constexpr bool SIDE_IN = Cfg::EPI_SIDE;
    static constexpr int BOX = Cfg::EPI_BOX;

    const GemmArgs& a;
    const EpiMaps<SIDE_IN>& maps;
    const AbortState& ab;
    uint8_t* const buf;          // two boxes
    float* const bias_s;         // 64 floats
    uint64_t* const bar;         // side box landed, per buffer
    const int quad, lane, half;
    uint32_t phases = 0;         // bit b: parity of the next wait for buffer b
    uint32_t pending = 0;        // bit b: a side box is on its way into buffer b
    float2 bias[2];              // of chunk 0 and 1, two columns per lane
    float gs = 0.0f;             // QUANT: gs_h

    // smem: the boxes of all epilogue warps (512-byte aligned, as their swizzle is), then their biases
    __device__ __forceinline__ EpiRows(const GemmArgs& args, const EpiMaps<SIDE_IN>& m, int q, int l, int h, uint8_t* smem,
                                       uint64_t* bars, const AbortState& abort)
        : a(args), maps(m), ab(abort), buf(smem + (4 * h + q) * Cfg::EPI_WARP),
          bias_s(reinterpret_cast<float*>(smem + kEpilogueWarps * Cfg::EPI_WARP + (4 * h + q) * Cfg::EPI_BIAS)),
          bar(bars + 2 * (4 * h + q)), quad(q), lane(l), half(h)
    {
        if constexpr (QUANT) gs = ld_written(a.gs_h);
    }

    // Chunks of the tile in this warp's order: the last columns of the tile first for the second
    // warpgroup (with SF_IN_ACC they hold the next tile's scales).
    __device__ __forceinline__ int chunk_col(const Tile& ti, int k) const
    {
        const int cols = Cfg::NARROW ? ti.q_span : Cfg::BN;
        return half ? cols - 64 * (k + 1) : 64 * k;
    }
    __device__ __forceinline__ int chunks(const Tile& ti) const { return (Cfg::NARROW ? ti.q_span : Cfg::BN) / 128; }

    // Boxes of the tile are numbered in the warp's order, `per_chunk` of them to a chunk; box u
    // starts at output column first_col (a column of h for the gated products).
    template <bool F32>
    __device__ __forceinline__ int first_col(const Tile& ti, int u) const
    {
        constexpr int per_chunk = (LINEAR ? 2 : 1) * (F32 ? 2 : 1);
        const int k = u / per_chunk;
        const int c = ti.q0 + chunk_col(ti, k);
        return (LINEAR ? c : c >> 1) + (u - k * per_chunk) * (F32 ? 16 : 32);
    }
    __device__ __forceinline__ int end_col() const { return LINEAR ? a.N : a.inter; }

    // Side box u into buffer b (free). Boxes wholly past the columns are not requested.
    template <bool F32>
    __device__ __forceinline__ void request(const Tile& ti, int u, int b)
    {
        const int n = first_col<F32>(ti, u);
        if (n >= end_col()) return;
        if (lane == 0) {
            mbar_arrive_expect_tx(&bar[b], BOX);
            tma_load_2d(buf + b * BOX, &maps.side, &bar[b], n * (F32 ? 4 : 2), ti.p0 + 32 * quad, l2_policy_evict_first());
        }
        pending |= 1u << b;
    }
    __device__ __forceinline__ bool landed(int b)
    {
        if (!(pending >> b & 1u)) return true;
        const bool ok = __all_sync(0xffffffffu, mbar_wait(&bar[b], phases >> b & 1u, ab, kErrEpiSide));
        if (ok) {
            phases ^= 1u << b;
            pending &= ~(1u << b);
        }
        return ok;
    }

    __device__ __forceinline__ bool active(const Tile& ti) const { return ti.p0 + 32 * quad < a.M; }

    // The tile's first two boxes.
    template <bool F32>
    __device__ __forceinline__ void request_first(const Tile& ti)
    {
        request<F32>(ti, 0, 0);
        if (LINEAR || F32 || chunks(ti) == 2) request<F32>(ti, 1, 1);
    }

    __device__ __forceinline__ void begin(const Tile& ti)
    {
        if (!active(ti)) return;
        if constexpr (LINEAR || GRAD) {
            if (a.side != nullptr) {
                if (a.out_dtype == kOutF32) request_first<true>(ti);
                else request_first<false>(ti);
            }
        }
        if constexpr (LINEAR) {
            if (a.bias != nullptr) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int n = ti.q0 + chunk_col(ti, k) + 2 * lane;
                    bias[k] = make_float2(0.0f, 0.0f);
                    if (k < chunks(ti) && n < a.N) bias[k] = ld_written(reinterpret_cast<const float2*>(a.bias + n));
                }
            }
        }
    }

    // The 16-byte piece e of this lane's row in buffer b.
    __device__ __forceinline__ uint32_t slot(int b, int e) const
    {
        return smem_u32(buf) + b * BOX + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4);
    }

    // NV side values of type DT from pieces e0 .. of buffer b.
    template <int32_t DT, int NV>
    __device__ __forceinline__ void get(int b, int e0, float* v) const
    {
        constexpr int PER = DT == kOutF32 ? 4 : 8;
#pragma unroll
        for (int e = 0; e < NV / PER; ++e) {
            const uint4 q = lds_u4(slot(b, e0 + e));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == kOutF32) {
                    v[e * PER + i] = __uint_as_float(w[i]);
                } else {
                    const float2 f = unpack_out16x2(w[i], DT);
                    v[e * PER + 2 * i] = f.x;
                    v[e * PER + 2 * i + 1] = f.y;
                }
            }
        }
    }

    // NV values to columns n .. of this lane's output row (`ld` columns, of which those below `end`
    // are to be written), in 32-byte sectors where the address allows.
    template <int32_t DT, int NV>
    __device__ __forceinline__ void store_row(const Tile& ti, int ld, int n, int end, const float* v) const
    {
        constexpr int PER = DT == kOutF32 ? 4 : 8, ESZ = 16 / PER;   // elements per 16-byte piece, bytes of one
        const int m = ti.p0 + 32 * quad + lane;
        if (m >= a.M) return;
        uint4 w[NV / PER];
#pragma unroll
        for (int e = 0; e < NV / PER; ++e) {
            const float* x = v + e * PER;
            if constexpr (DT == kOutF32)
                w[e] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            else
                w[e] = make_uint4(pack_out16x2(x[0], x[1], DT), pack_out16x2(x[2], x[3], DT), pack_out16x2(x[4], x[5], DT),
                                  pack_out16x2(x[6], x[7], DT));
        }
        uint8_t* p = static_cast<uint8_t*>(a.out) + (static_cast<size_t>(m) * ld + n) * ESZ;
        if (((reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(ld) * ESZ) & 31) == 0) {
#pragma unroll
            for (int e = 0; e < NV / PER; e += 2)
                if (n + e * PER < end) st_global_32(p + 16 * e, w[e], w[e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < NV / PER; ++e)
                if (n + e * PER < end) *reinterpret_cast<uint4*>(p + 16 * e) = w[e];
        }
    }

    // Piece h (32 columns, r) of chunk k: one box of a 16-bit type, two of fp32.
    template <int32_t DT, bool SIDE>
    __device__ __forceinline__ bool linear_piece(const Tile& ti, int k, int h, const uint32_t (&r)[32], float alpha)
    {
        constexpr bool F32 = DT == kOutF32;
        constexpr int BOXES = F32 ? 2 : 1, NV = 32 / BOXES;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
        linear_act(a.bias != nullptr ? bias_s + 32 * h : nullptr, a.act_fn, alpha, v);
#pragma unroll
        for (int s = 0; s < BOXES; ++s) {
            const int u = BOXES * (2 * k + h) + s, b = u & 1;
            if constexpr (SIDE) {
                if (!landed(b)) return false;
                float x[NV];
                get<DT, NV>(b, 0, x);
                __syncwarp();
                if (u + 2 < 2 * BOXES * chunks(ti)) request<F32>(ti, u + 2, b);
                const f32x2 sc = pack2(a.side_scale, a.side_scale);
#pragma unroll
                for (int i = 0; i < NV; i += 2) {
                    float* w = v + NV * s + i;
                    unpack2(fma2(sc, pack2(x[i], x[i + 1]), pack2(w[0], w[1])), w[0], w[1]);
                }
            }
            store_row<DT, NV>(ti, a.N, first_col<F32>(ti, u), a.N, v + NV * s);
        }
        return true;
    }

    // 16 indices of h from [16 gate, 16 up] columns: half a box of a 16-bit type, one of fp32.
    template <int32_t DT>
    __device__ __forceinline__ bool glu_piece(const Tile& ti, int k, int h, const uint32_t (&r)[32], float alpha,
                                              uint32_t (&q)[4], uint32_t& sf)
    {
        constexpr bool F32 = DT == kOutF32;
        const int e0 = F32 ? 0 : 2 * h, u = F32 ? 2 * k + h : k;
        const f32x2 al = pack2(alpha, alpha);
        float g[16], w[16];                          // g and u
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            unpack2(mul2(al, pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1]))), g[i], g[i + 1]);
            unpack2(mul2(al, pack2(__uint_as_float(r[16 + i]), __uint_as_float(r[17 + i]))), w[i], w[i + 1]);
        }
        const int j = ((ti.q0 + chunk_col(ti, k)) >> 1) + 16 * h;    // first index of h
        if constexpr (GRAD) {
            const int b = u & 1;
            float d[16], x[16];
            if (!landed(b)) return false;
            get<DT, 16>(b, e0, x);
            if (F32 || h == 1) {
                __syncwarp();
                if (u + 2 < (F32 ? 2 : 1) * chunks(ti)) request<F32>(ti, u + 2, b);
            }
            act_apply_grad(g, d, a.act_fn);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const f32x2 s = pack2(x[i], x[i + 1]);
                unpack2(mul2(mul2(pack2(d[i], d[i + 1]), pack2(w[i], w[i + 1])), s), d[i], d[i + 1]);
                unpack2(mul2(pack2(g[i], g[i + 1]), s), g[i], g[i + 1]);
            }
            if (j < a.inter) {
                store_row<DT, 16>(ti, a.N, j, a.N, d);
                store_row<DT, 16>(ti, a.N, a.inter + j, a.N, g);
            }
            return true;
        }
        act_apply(g, a.act_fn);
#pragma unroll
        for (int i = 0; i < 16; i += 2) unpack2(mul2(pack2(g[i], g[i + 1]), pack2(w[i], w[i + 1])), g[i], g[i + 1]);
        if constexpr (QUANT) {
            // one NVFP4 block per piece; a row's two blocks of a chunk leave together
            float amax = 0.0f, rcp, lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(g[i]));
            const uint32_t s = block_scale(amax, gs, rcp);
#pragma unroll
            for (int i = 0; i < 8; ++i) { lo[i] = g[i]; hi[i] = g[8 + i]; }
            q[2] = scale_to_e2m1x8(lo, rcp);
            q[3] = scale_to_e2m1x8(hi, rcp);
            if (h == 0) {
                q[0] = q[2];
                q[1] = q[3];
                sf = s;
            } else {
                const int m = ti.p0 + 32 * quad + lane;
                if (m < a.M && j < a.inter) {
                    *reinterpret_cast<uint4*>(a.h_q + static_cast<int64_t>(m) * (a.inter >> 1) + ((j - 16) >> 1)) =
                        make_uint4(q[0], q[1], q[2], q[3]);
                    *reinterpret_cast<uint16_t*>(h_sf_at(a, m, (j >> 4) - 1)) = static_cast<uint16_t>(sf | s << 8);
                }
            }
        } else {
            store_row<DT, 16>(ti, a.inter, j, a.inter, g);
        }
        return true;
    }

    // Drains the tile from TMEM (tacc: this warp's lanes and the accumulator's first column);
    // `drained` is called once the first chunk is in registers. The output type and the side
    // input are decided once per tile: branches inside would cut the code into blocks too short
    // to hide its latencies with two warps to a scheduler.
    template <int32_t DT, bool SIDE, class F>
    __device__ __forceinline__ bool finish_as(const Tile& ti, uint32_t tacc, float alpha, F drained)
    {
        uint32_t q[4], sf = 0;
        bool ok = true;
        const int nk = chunks(ti);
#pragma unroll 1
        for (int k = 0; k < nk; ++k) {
            uint32_t r[4][16], cur[32];
            const uint32_t t0 = tacc + chunk_col(ti, k);
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x16(t0 + 16 * i, r[i]);
            if constexpr (LINEAR) {
                if (a.bias != nullptr) {
                    __syncwarp();                    // the chunk before has read its bias
                    reinterpret_cast<float2*>(bias_s)[lane] = k == 0 ? bias[0] : bias[1];
                    __syncwarp();
                }
            }
            tmem_ld_wait();
            if (k == 0) drained();
#pragma unroll
            for (int i = 0; i < 32; ++i) cur[i] = r[i >> 4][i & 15];
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if constexpr (LINEAR) ok = ok && linear_piece<DT, SIDE>(ti, k, h, cur, alpha);
                else ok = ok && glu_piece<DT>(ti, k, h, cur, alpha, q, sf);
#pragma unroll
                for (int i = 0; i < 32; ++i) cur[i] = r[2 + (i >> 4)][i & 15];
            }
        }
        return __all_sync(0xffffffffu, ok);
    }

    template <int32_t DT, class F>
    __device__ __forceinline__ bool finish_type(const Tile& ti, uint32_t tacc, float alpha, F drained)
    {
        if constexpr (LINEAR) {
            if (a.side == nullptr) return finish_as<DT, false>(ti, tacc, alpha, drained);
        }
        return finish_as<DT, true>(ti, tacc, alpha, drained);
    }

    template <class F>
    __device__ __forceinline__ bool finish(const Tile& ti, uint32_t tacc, float alpha, F drained)
    {
        if (!active(ti)) {
            drained();
            return true;
        }
        if constexpr (!QUANT) {
            if (a.out_dtype == kOutF32) return finish_type<kOutF32>(ti, tacc, alpha, drained);
            if (a.out_dtype == kOutF16) return finish_type<kOutF16>(ti, tacc, alpha, drained);
        }
        return finish_type<kOutBF16>(ti, tacc, alpha, drained);
    }

    // Before the CTA's shared memory is released: every box has landed.
    __device__ __forceinline__ void drain()
    {
        for (int b = 0; b < 2; ++b)
            if (pending >> b & 1u) mbar_wait_drain(&bar[b], phases >> b & 1u);
    }
};

}  // namespace nvfp4
