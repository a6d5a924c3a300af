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

// 1 / (1 + exp(-x)); exp overflows to infinity for x < -88.7, where the quotient is 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + expf(-x)); }

// p = sigmoid(x) and q = 1 - p = p exp(-x), each to a few ulp (1 - p itself would lose q where p is
// near 1). The exponent is capped, where p is already negligible, so that exp stays finite.
__device__ __forceinline__ void sigmoid_both(float x, float& p, float& q)
{
    const float e = expf(fminf(-x, 80.0f));
    p = __fdividef(1.0f, 1.0f + e);
    q = p * e;
}

// 2 sqrt(2 / pi) (x + 0.044715 x^3): gelu_tanh(x) = x sigmoid(this), since
// (1 + tanh z) / 2 = sigmoid(2 z).
constexpr float kGeluC = 1.5957691216057308f, kGeluA = 0.044715f;

// v = act(v) for all elements (the switch is uniform, one branch per array).
template <int N>
__device__ __forceinline__ void act_apply(float (&v)[N], int32_t act)
{
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
            for (int i = 0; i < N; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(v[i] * 0.70710678118654752f));
            break;
        case kActGeluTanh:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= sigmoid(kGeluC * v[i] * fmaf(kGeluA * v[i], v[i], 1.0f));
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= sigmoid(v[i]);
            break;
        default: break;
    }
}

// v = act(v) and d = act'(v) (0 at the kink of relu and relu2).
template <int N>
__device__ __forceinline__ void act_apply_grad(float (&v)[N], float (&d)[N], int32_t act)
{
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
            for (int i = 0; i < N; ++i) {
                const float x = v[i];
                const float cdf = 0.5f * (1.0f + erff(x * 0.70710678118654752f));
                d[i] = fmaf(x, 0.3989422804014327f * expf(-0.5f * x * x), cdf);
                v[i] = x * cdf;
            }
            break;
        case kActGeluTanh:
            // p + x p q z'(x), p = sigmoid(z), q = 1 - p, z = C x (1 + A x^2); x^2 is capped where
            // p q is already 0, so that an overflowing z' cannot make 0 * infinity
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = v[i];
                float p, q;
                sigmoid_both(kGeluC * x * fmaf(kGeluA * x, x, 1.0f), p, q);
                const float dz = kGeluC * fmaf(3.0f * kGeluA, fminf(x * x, 1e8f), 1.0f);
                d[i] = fmaf(x * (p * q), dz, p);
                v[i] = x * p;
            }
            break;
        case kActSilu:
            // p + x p q
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float x = v[i];
                float p, q;
                sigmoid_both(x, p, q);
                d[i] = fmaf(x * p, q, p);
                v[i] = x * p;
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
// is read with plain loads, each element by the thread that later writes its place.
__device__ __forceinline__ float load_side1(const GemmArgs& a, size_t idx)
{
    if (a.out_dtype == kOutF32) return static_cast<const float*>(a.side)[idx];
    const uint32_t w = static_cast<const uint16_t*>(a.side)[idx];
    return unpack_out16x2(w, a.out_dtype).x;
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

// A 4 x 4 transpose of 16-byte chunks within each group of 4 lanes (transpose_chunks8 for rows of
// 64 bytes): lane 4 g + j leaves with chunk j of rows 4 g .. 4 g + 3. Its own inverse.
__device__ __forceinline__ void transpose_chunks4(uint32_t (&w)[4][4], int lane)
{
    const int j = lane & 3;
#pragma unroll
    for (int m = 2; m >= 1; m >>= 1) {
        const bool hi = (j & m) != 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (e & m) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t send = hi ? w[e][k] : w[e ^ m][k];
                const uint32_t recv = __shfl_xor_sync(0xffffffffu, send, m);
                if (hi) w[e][k] = recv;
                else w[e ^ m][k] = recv;
            }
        }
    }
}

// 32 consecutive elements (columns col .. col + 31 of a row-major array with row stride ld) of
// each of the warp's 32 rows row0 + lane, one row per lane in registers, moved as 64-byte
// (16-bit types) or 128-byte (fp32) row segments: a transpose among 4 or 8 lanes turns each
// lane's row into the chunk it loads or stores of 4 or 8 rows. Rows from M and columns from
// n_end (a multiple of 8) on are not touched; they load as 0.
__device__ __forceinline__ void load_rows32(const void* src, int32_t dt, int64_t ld, int row0, int M, int col,
                                            int n_end, int lane, float (&v)[32])
{
    if (dt == kOutF32) {
        const int n = col + 4 * (lane & 7);
        uint32_t w[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int m = row0 + (lane & ~7) + t;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (m < M && n < n_end) x = *reinterpret_cast<const uint4*>(static_cast<const float*>(src) + m * ld + n);
            w[t][0] = x.x; w[t][1] = x.y; w[t][2] = x.z; w[t][3] = x.w;
        }
        transpose_chunks8(w, lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(w[i >> 2][i & 3]);
    } else {
        const int n = col + 8 * (lane & 3);
        uint32_t w[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int m = row0 + (lane & ~3) + t;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (m < M && n < n_end) x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + m * ld + n);
            w[t][0] = x.x; w[t][1] = x.y; w[t][2] = x.z; w[t][3] = x.w;
        }
        transpose_chunks4(w, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 f = unpack_out16x2(w[i >> 2][i & 3], dt);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void store_rows32(void* dst, int32_t dt, int64_t ld, int row0, int M, int col, int lane,
                                             const float (&v)[32])
{
    if (dt == kOutF32) {
        uint32_t w[8][4];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i >> 2][i & 3] = __float_as_uint(v[i]);
        transpose_chunks8(w, lane);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int m = row0 + (lane & ~7) + t;
            if (m < M)
                *reinterpret_cast<uint4*>(static_cast<float*>(dst) + m * ld + col + 4 * (lane & 7)) =
                    make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        }
    } else {
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = pack_out16x2(v[2 * i], v[2 * i + 1], dt);
        transpose_chunks4(w, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int m = row0 + (lane & ~3) + t;
            if (m < M)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + m * ld + col + 8 * (lane & 3)) =
                    make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
        }
    }
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

// v = act(alpha * acc + bias) of N consecutive output columns n0 .. of one row (N a multiple of
// 8; columns past a.N read no bias, N % 8 == 0 of the output).
template <int N>
__device__ __forceinline__ void linear_act(const GemmArgs& a, int n0, float alpha, float (&v)[N])
{
    if (a.bias != nullptr) {
#pragma unroll
        for (int k = 0; k < N; k += 4) {
            float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (n0 + k < a.N) b = __ldg(reinterpret_cast<const float4*>(a.bias + n0 + k));
            v[k] = fmaf(alpha, v[k], b.x);
            v[k + 1] = fmaf(alpha, v[k + 1], b.y);
            v[k + 2] = fmaf(alpha, v[k + 2], b.z);
            v[k + 3] = fmaf(alpha, v[k + 3], b.w);
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] *= alpha;
    }
    act_apply(v, a.act_fn);
}

template <class Cfg>
__device__ __forceinline__ void linear_rows64(const GemmArgs& a, const Tile& ti, int quad, int lane, int c0,
                                              const uint32_t (&r)[4][16], float alpha)
{
    const int row0 = ti.p0 + 32 * quad;
    uint32_t o[4][16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n0 = ti.q0 + c0 + 32 * h;
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[2 * h + (i >> 4)][i & 15]);
        linear_act(a, n0, alpha, v);
        if (a.side != nullptr) {
            float s[32];
            load_rows32(a.side, a.out_dtype, a.N, row0, a.M, n0, a.N, lane, s);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(a.side_scale, s[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[2 * h + (i >> 4)][i & 15] = __float_as_uint(v[i]);
    }
    store_rows64<Cfg>(a, ti, quad, lane, c0, o, 1.0f);
}

// Swap tiles: the lane's output column n = p0 + 32 quad + lane, tokens c .. c + 15.
template <class Cfg>
__device__ __forceinline__ void linear_tok16(const GemmArgs& a, const Tile& ti, int quad, int lane, int c,
                                             const uint32_t (&r)[16], float alpha)
{
    const int n = ti.p0 + 32 * quad + lane;
    const float b = a.bias != nullptr && n < a.N ? __ldg(a.bias + n) : 0.0f;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = fmaf(alpha, __uint_as_float(r[j]), b);
    act_apply(v, a.act_fn);
    if (a.side != nullptr) {
        float s[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int m = ti.q0 + c + j;
            s[j] = m < a.M && n < a.N ? load_side1(a, static_cast<size_t>(m) * a.N + n) : 0.0f;
        }
        // (the 16-bit stores below go to other columns than this lane's: every lane has its
        // residuals before any lane of the warp stores, and no other warp has these columns)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = fmaf(a.side_scale, s[j], v[j]);
        __syncwarp();
    }
    uint32_t o[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(v[j]);
    if (a.out_dtype != kOutF32) store_tok16<Cfg>(a, ti, quad, lane, c, o, 1.0f);
    else store_out16<Cfg>(a, ti, n, c, o, 1.0f);
}

// A reduced split-K chunk (see store_chunk): eight consecutive outputs per item.
template <class Cfg>
__device__ __forceinline__ void linear_chunk(const GemmArgs& a, const Tile& ti, const float* src, int nsrc, int r0,
                                             int rows, int tid, float alpha)
{
    constexpr int BN = Cfg::BN;
    constexpr int PS = Cfg::PSTRIDE;
    const int G = Cfg::SWAP ? rows >> 3 : BN / 8;
    const int items = Cfg::SWAP ? BN * G : rows * G;
    for (int item = tid; item < items; item += 128) {
        const int outer = item / G, inner = (item - outer * G) * 8;
        // swap: outer = token column, inner = chunk row; otherwise outer = chunk row, inner = column
        const int m = Cfg::SWAP ? ti.q0 + outer : ti.p0 + r0 + outer;
        const int n0 = Cfg::SWAP ? ti.p0 + r0 + inner : ti.q0 + inner;
        if (m >= a.M || n0 >= a.N) continue;
        const size_t idx = static_cast<size_t>(m) * a.N + n0;
        float s[8];
        if (a.side != nullptr) load_side(a, idx, s);          // in flight during the sums
        float v[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = 0.0f;
        for (int j = 0; j < nsrc; ++j) {
            if constexpr (Cfg::SWAP) {
                const float* p = src + (j * rows + inner) * PS + outer;
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] += p[t * PS];
            } else {
                const float* p = src + (j * rows + outer) * PS + inner;
#pragma unroll
                for (int t = 0; t < 8; t += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(p + t);
                    v[t] += x.x; v[t + 1] += x.y; v[t + 2] += x.z; v[t + 3] += x.w;
                }
            }
        }
        linear_act(a, n0, alpha, v);
        if (a.side != nullptr) {
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = fmaf(a.side_scale, s[t], v[t]);
        }
        store_out8(a, idx, v);
    }
}

// ------------------------------------------------------------------ gated product

// Token-major tiles: columns c0 .. c0 + 63 are [16 gate, 16 up, 16 gate, 16 up] of 32 indices of
// h, all in the thread of their token (I % 32 == 0: the 32 are inside I or past it together).
template <class Cfg>
__device__ __forceinline__ void glu_rows64(const GemmArgs& a, const Tile& ti, int quad, int lane, int c0,
                                           const uint32_t (&r)[4][16], float alpha)
{
    const int j0 = (ti.q0 + c0) >> 1;
    if (j0 >= a.inter) return;                       // warp-uniform
    const int row0 = ti.p0 + 32 * quad;
    float h[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = alpha * __uint_as_float(r[2 * (i >> 4)][i & 15]);
    if constexpr (Cfg::EPI == kEpiGluGrad) {
        float s[32], d[32];
        load_rows32(a.side, a.out_dtype, a.inter, row0, a.M, j0, a.inter, lane, s);
        act_apply_grad(h, d, a.act_fn);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float u = alpha * __uint_as_float(r[2 * (i >> 4) + 1][i & 15]);
            d[i] = s[i] * u * d[i];
            h[i] = s[i] * h[i];
        }
        store_rows32(a.out, a.out_dtype, a.N, row0, a.M, j0, lane, d);
        store_rows32(a.out, a.out_dtype, a.N, row0, a.M, a.inter + j0, lane, h);
    } else {
        act_apply(h, a.act_fn);
#pragma unroll
        for (int i = 0; i < 32; ++i) h[i] *= alpha * __uint_as_float(r[2 * (i >> 4) + 1][i & 15]);
        if constexpr (Cfg::EPI == kEpiGlu) {
            store_rows32(a.out, a.out_dtype, a.inter, row0, a.M, j0, lane, h);
        } else {
            const float gs = __ldg(a.gs_h);
            uint32_t q[4], sf = 0;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float amax = 0.0f, rcp, lo[8], hi[8];
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(h[16 * b + i]));
                sf |= block_scale(amax, gs, rcp) << (8 * b);
#pragma unroll
                for (int i = 0; i < 8; ++i) { lo[i] = h[16 * b + i]; hi[i] = h[16 * b + 8 + i]; }
                q[2 * b] = scale_to_e2m1x8(lo, rcp);
                q[2 * b + 1] = scale_to_e2m1x8(hi, rcp);
            }
            const int m = row0 + lane;
            if (m < a.M) {
                // 16 bytes of codes and two neighbouring scale bytes (an even block index)
                *reinterpret_cast<uint4*>(a.h_q + static_cast<int64_t>(m) * (a.inter >> 1) + (j0 >> 1)) =
                    make_uint4(q[0], q[1], q[2], q[3]);
                *reinterpret_cast<uint16_t*>(h_sf_at(a, m, j0 >> 4)) = static_cast<uint16_t>(sf);
            }
        }
    }
}

// One (g, u) pair of h index j of token m, after the reduction; the 16 lanes of a half-warp hold
// the 16 indices of one block of the same token. `ok`: the token exists. All lanes take part.
template <class Cfg>
__device__ __forceinline__ void glu_lane(const GemmArgs& a, int m, int j, float g, float u, bool ok)
{
    float v[1] = {g};
    if constexpr (Cfg::EPI == kEpiGluGrad) {
        float d[1];
        act_apply_grad(v, d, a.act_fn);
        if (ok) {
            const float s = load_side1(a, static_cast<size_t>(m) * a.inter + j);
            const size_t idx = static_cast<size_t>(m) * a.N + j;
            store_out1(a, idx, s * u * d[0]);
            store_out1(a, idx + a.inter, s * v[0]);
        }
    } else {
        act_apply(v, a.act_fn);
        const float h = v[0] * u;
        if constexpr (Cfg::EPI == kEpiGlu) {
            if (ok) store_out1(a, static_cast<size_t>(m) * a.inter + j, h);
        } else {
            float amax = fabsf(h), rcp;
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t sf = block_scale(amax, __ldg(a.gs_h), rcp);
            const uint32_t code = f32x2_to_e2m1x2(__fmul_rn(h, rcp), 0.0f) & 0xFu;
            const uint32_t next = __shfl_xor_sync(0xffffffffu, code, 1);
            if (ok && (j & 1) == 0)
                a.h_q[static_cast<int64_t>(m) * (a.inter >> 1) + (j >> 1)] = static_cast<uint8_t>(code | (next << 4));
            if (ok && (j & 15) == 0) *h_sf_at(a, m, j >> 4) = static_cast<uint8_t>(sf);
        }
    }
}

// Weight-major tiles: lanes 0-15 hold 16 gate rows and lanes 16-31 their up rows, for tokens
// c .. c + 15. One exchange gives lane i (i < 16) both halves of tokens c .. c + 7 and lane
// 16 + i those of tokens c + 8 .. c + 15.
template <class Cfg>
__device__ __forceinline__ void glu_tok16(const GemmArgs& a, const Tile& ti, int quad, int lane, int c,
                                          const uint32_t (&r)[16], float alpha)
{
    const int j0 = (ti.p0 >> 1) + 16 * quad;
    if (j0 >= a.inter) return;                       // warp-uniform
    const bool up = lane >= 16;
#pragma unroll
    for (int cc = 0; cc < 8; ++cc) {
        const float lo = alpha * __uint_as_float(r[cc]);        // token c + cc
        const float hi = alpha * __uint_as_float(r[cc + 8]);    // token c + 8 + cc
        const float other = __shfl_xor_sync(0xffffffffu, up ? lo : hi, 16);
        const int m = ti.q0 + c + cc + (up ? 8 : 0);
        glu_lane<Cfg>(a, m, j0 + (lane & 15), up ? other : lo, up ? hi : other, m < a.M);
    }
}

// A reduced split-K chunk. Weight-major: item = (32-row group, token, index of the group), so that
// a half-warp has one block of one token. Token-major: item = (chunk row, four indices of h); the
// four lanes of a block are neighbours. The item count is a multiple of 128 either way: every
// lane of a warp stays in the loop for its exchanges.
template <class Cfg>
__device__ __forceinline__ void glu_chunk(const GemmArgs& a, const Tile& ti, const float* src, int nsrc, int r0,
                                          int rows, int tid, float alpha)
{
    constexpr int BN = Cfg::BN;
    constexpr int PS = Cfg::PSTRIDE;
    if constexpr (Cfg::SWAP) {
        for (int item = tid; item < (rows >> 5) * BN * 16; item += 128) {
            const int i = item & 15, c = (item >> 4) % BN, unit = (item >> 4) / BN;
            const float* p = src + (32 * unit + i) * PS + c;
            float g = 0.0f, u = 0.0f;
            for (int k = 0; k < nsrc; ++k) {
                g += p[k * rows * PS];
                u += p[(k * rows + 16) * PS];
            }
            const int j = ((ti.p0 + r0) >> 1) + 16 * unit + i, m = ti.q0 + c;
            glu_lane<Cfg>(a, m, j, alpha * g, alpha * u, m < a.M && j < a.inter);
        }
    } else {
        constexpr int G = BN / 8;                    // items per row: four indices of h each
        static_assert(G % 4 == 0 && G * 8 % 128 == 0, "whole warps of items (chunks are multiples of 8 rows)");
        for (int item = tid; item < rows * G; item += 128) {
            const int lr = item / G, cg = (item % G) >> 2, s = item & 3;
            const float* p = src + lr * PS + 32 * cg + 4 * s;
            float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = 0; k < nsrc; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(p + k * rows * PS);
                const float4 y = *reinterpret_cast<const float4*>(p + k * rows * PS + 16);
                g[0] += x.x; g[1] += x.y; g[2] += x.z; g[3] += x.w;
                u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) { g[i] *= alpha; u[i] *= alpha; }
            const int m = ti.p0 + r0 + lr, j = ((ti.q0 + 32 * cg) >> 1) + 4 * s;
            const bool ok = m < a.M && j < a.inter;
            if constexpr (Cfg::EPI == kEpiGluGrad) {
                float d[4], dh[4];
                if (!ok) continue;                   // no exchange below
                load_side(a, static_cast<size_t>(m) * a.inter + j, dh);
                act_apply_grad(g, d, a.act_fn);
#pragma unroll
                for (int i = 0; i < 4; ++i) { d[i] = dh[i] * u[i] * d[i]; g[i] = dh[i] * g[i]; }
                const size_t idx = static_cast<size_t>(m) * a.N + j;
                store_out4(a, idx, d);
                store_out4(a, idx + a.inter, g);
            } else {
                act_apply(g, a.act_fn);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] *= u[i];
                if constexpr (Cfg::EPI == kEpiGlu) {
                    if (ok) store_out4(a, static_cast<size_t>(m) * a.inter + j, g);
                } else {
                    float amax = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3]))), rcp;
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    const uint32_t sf = block_scale(amax, __ldg(a.gs_h), rcp);
                    const uint32_t q = f32x2_to_e2m1x2(__fmul_rn(g[0], rcp), __fmul_rn(g[1], rcp)) |
                                       f32x2_to_e2m1x2(__fmul_rn(g[2], rcp), __fmul_rn(g[3], rcp)) << 8;
                    if (ok) {
                        *reinterpret_cast<uint16_t*>(a.h_q + static_cast<int64_t>(m) * (a.inter >> 1) + (j >> 1)) =
                            static_cast<uint16_t>(q);
                        if (s == 0) *h_sf_at(a, m, j >> 4) = static_cast<uint8_t>(sf);
                    }
                }
            }
        }
    }
}

// ------------------------------------------------------------------ dispatch (gemm_kernel.cuh)

template <class Cfg>
__device__ __forceinline__ void epi_rows64(const GemmArgs& a, const Tile& ti, int quad, int lane, int c0,
                                           const uint32_t (&r)[4][16], float alpha)
{
    if constexpr (Cfg::EPI == kEpiLinear) linear_rows64<Cfg>(a, ti, quad, lane, c0, r, alpha);
    else glu_rows64<Cfg>(a, ti, quad, lane, c0, r, alpha);
}

template <class Cfg>
__device__ __forceinline__ void epi_tok16(const GemmArgs& a, const Tile& ti, int quad, int lane, int c,
                                          const uint32_t (&r)[16], float alpha)
{
    if constexpr (Cfg::EPI == kEpiLinear) linear_tok16<Cfg>(a, ti, quad, lane, c, r, alpha);
    else glu_tok16<Cfg>(a, ti, quad, lane, c, r, alpha);
}

template <class Cfg>
__device__ __forceinline__ void epi_chunk(const GemmArgs& a, const Tile& ti, const float* src, int nsrc, int r0,
                                          int rows, int tid, float alpha)
{
    if constexpr (Cfg::EPI == kEpiLinear) linear_chunk<Cfg>(a, ti, src, nsrc, r0, rows, tid, alpha);
    else glu_chunk<Cfg>(a, ti, src, nsrc, r0, rows, tid, alpha);
}

}  // namespace nvfp4
