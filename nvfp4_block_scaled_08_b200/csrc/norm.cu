// norm.cu -- the residual add and the norms around a transformer block in one pass, with a 16- or
// 32-bit or an NVFP4 output (nvfp4_residual_norm, nvfp4_residual_norm_quantize).
//
// Per row, with N(z) = z / sqrt(mean(z^2) + eps) (RMS) or (z - mean z) / sqrt(var z + eps) (layer):
//     v = y;  v = N(v) * post_weight;  v = gate * v            (the last two optional)
//     r = T(x + residual_scale * v)                            (r = x without y; T: x's type)
//     n = N(r) * weight (+ bias)
// and n is rounded once to the output type, or quantised as nvfp4_quantize does with a fixed
// global scale.
//
// HBM-bound: x and y are read once, r and the output written once, a few tens of fp32 operations
// per element. So a row stays in registers from its load to its last store (8 V elements per
// thread), and all loads of a row are in flight before its first reduction. Sums are fp32 in a
// fixed order: 8 V elements per thread, then butterflies in the warp and over the warps; the
// layer norm's variance is a second sum over the centred values (no E[z^2] - E[z]^2).
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "quant_core.cuh"

namespace nvfp4 {

namespace {

// 16-byte load that leaves no line in L1 (rows are read once; the weights stay there). Not the
// read-only path: r may be written over x or y, and the kernel before may have written both.
__device__ __forceinline__ uint4 load16(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Eight fp32 values (a lane's 32 bytes beside the next lane's) as one access where the address
// allows (`wide`: 32-byte aligned), else as two: two 16-byte accesses 32 bytes apart use half of
// each 128-byte line that they pass L1 with.
__device__ __forceinline__ void load32(const float* p, bool wide, uint4& lo, uint4& hi)
{
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
                     : "l"(p)
                     : "memory");
    } else {
        lo = load16(p);
        hi = load16(p + 4);
    }
}

// Eight consecutive elements as they sit in memory, and their values.
template <typename T> struct Vec8;
template <> struct Vec8<float> {
    uint4 lo, hi;
    __device__ void load(const float* p, bool wide) { load32(p, wide, lo, hi); }
    __device__ void store(float* p, bool wide) const
    {
        if (wide) {
            st_global_32(p, lo, hi);
        } else {
            reinterpret_cast<uint4*>(p)[0] = lo;
            reinterpret_cast<uint4*>(p)[1] = hi;
        }
    }
    __device__ void decode(float (&v)[8]) const { InTraits<float>::decode(Raw32{lo, hi}, v); }
    __device__ void encode(const float (&v)[8])
    {
        lo = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        hi = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    }
};
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ void load(const __nv_bfloat16* p, bool) { u = load16(p); }
    __device__ void store(__nv_bfloat16* p, bool) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ void decode(float (&v)[8]) const { InTraits<__nv_bfloat16>::decode(u, v); }
    __device__ void encode(const float (&v)[8])
    {
        u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
};
template <> struct Vec8<__half> {
    uint4 u;
    __device__ void load(const __half* p, bool) { u = load16(p); }
    __device__ void store(__half* p, bool) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ void decode(float (&v)[8]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    __device__ void encode(const float (&v)[8])
    {
        u = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
    }
};

template <typename T>
__device__ __forceinline__ void store_as(void* out, int64_t idx, const float (&v)[8], bool wide)
{
    Vec8<T> w;
    w.encode(v);
    w.store(static_cast<T*>(out) + idx, wide);
}

// Eight weights. p is behind_wait(): the kernel before may have written them (a gate that it
// worked out, say), so they are neither constant data nor free to be loaded before the wait; behind
// it the compiler may place the loads as it likes (no output overlaps them).
__device__ __forceinline__ void load_weights(const float* p, float (&v)[8], bool wide)
{
    if (wide) {
        asm("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
            : "l"(p));
    } else {
        asm("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
        asm("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p + 4));
    }
}

// Sum over the TPR threads of a row, in a fixed order. `red` holds two slots of TPR / 32 floats,
// used in turn (`slot`), so that one barrier per sum suffices: a slot is written again only
// after the barrier of the sum in between.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float* red, int& slot)
{
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float* mine = red + slot * W;
        slot ^= 1;
        if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = s;
        __syncthreads();
        s = mine[threadIdx.x & (W - 1)];
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    return s;
}

// z = N(z) for the row's values z[V][8]; vectors past the row (`in` false) are 0 and stay 0.
template <int TPR, int V>
__device__ __forceinline__ void normalise(const NormLaunch& a, float (&z)[V][8], const bool (&in)[V], float* red,
                                          int& slot)
{
    if (a.layer) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += z[k][i];
        const float mean = row_sum<TPR>(s, red, slot) * a.inv_h;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (in[k]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[k][i] -= mean;
            }
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(z[k][i], z[k][i], s);
    const float rstd = __frsqrt_rn(fmaf(row_sum<TPR>(s, red, slot), a.inv_h, a.eps));
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[k][i] *= rstd;
}

// z *= weights of its columns
template <int TPR, int V>
__device__ __forceinline__ void multiply(float (&z)[V][8], const bool (&in)[V], int t, const float* weights, bool wide)
{
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if (!in[k]) continue;
        float w[8];
        load_weights(weights + 8 * (t + k * TPR), w, wide);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[k][i] *= w[i];
    }
}

// One row per TPR threads; thread t holds the row's 8-element vectors t, t + TPR, ... (V of them).
// What bounds it: HBM without post_weight and gate (16384 x 6144 bf16: 122 us, 6.6 TB/s); with
// them (140 us) the second chain of sum and barrier, and the fp32 weights, which pass L1 for
// every row. Two rows to a block share the weights but keep fewer rows on an SM (160 us); so do
// blocks that walk several rows with the next row's loads ahead (138 us where this takes 122).
template <typename T, int TPR, int V, bool QUANT>
__global__ void __launch_bounds__(TPR <= 32 ? 128 : TPR) residual_norm_kernel(const NormLaunch a)
{
    __shared__ float red[TPR > 32 ? 2 * (TPR / 32) : 1];
    const int t = threadIdx.x % TPR;
    const int64_t row = TPR <= 32 ? blockIdx.x * static_cast<int64_t>(blockDim.x / TPR) + threadIdx.x / TPR : blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const float *w_n = behind_wait(a.w), *b_n = behind_wait(a.b), *w_post = behind_wait(a.post), *w_gate = behind_wait(a.gate);
    // rows past the last one (TPR <= 32) hold nothing, but stay for their warp's exchanges
    const int nvec = row < a.rows ? a.H >> 3 : 0;
    const bool wide = a.wide != 0;
    int slot = 0;
    bool in[V];
    Vec8<T> xw[V], yw[V];
    const T* x = static_cast<const T*>(a.x) + row * a.ld_x;
    const T* y = static_cast<const T*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = t + k * TPR;
        in[k] = c < nvec;
        xw[k] = Vec8<T>{};
        yw[k] = Vec8<T>{};
        if (in[k]) {
            xw[k].load(x + 8 * c, wide);
            if (a.y) yw[k].load(y + 8 * c, wide);
        }
    }
    float z[V][8];
    if (a.y) {
#pragma unroll
        for (int k = 0; k < V; ++k) yw[k].decode(z[k]);
        if (a.post) {
            normalise<TPR, V>(a, z, in, red, slot);
            multiply<TPR, V>(z, in, t, w_post, wide);
        }
        if (a.gate) multiply<TPR, V>(z, in, t, w_gate, wide);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!in[k]) continue;
            float xv[8];
            xw[k].decode(xv);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[k][i] = fmaf(a.scale, z[k][i], xv[i]);
            // the next norm is of the residual as it is stored: what a separate norm would read
            xw[k].encode(z[k]);
            xw[k].decode(z[k]);
            if (a.r) xw[k].store(static_cast<T*>(a.r) + row * a.ld_r + 8 * (t + k * TPR), wide);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) xw[k].decode(z[k]);
    }
    normalise<TPR, V>(a, z, in, red, slot);
    const float gs = QUANT ? ld_written(a.gs) : 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = t + k * TPR;
        if (in[k]) {
            float w[8];
            load_weights(w_n + 8 * c, w, wide);
            if (a.b) {
                float b[8];
                load_weights(b_n + 8 * c, b, wide);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[k][i] = fmaf(z[k][i], w[i], b[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[k][i] *= w[i];
            }
        }
        if constexpr (!QUANT) {
            if (!in[k]) continue;
            const int64_t idx = row * a.H + 8 * c;
            if (a.out_dt == 2) store_as<float>(a.out, idx, z[k], wide);
            else if (a.out_dt == 1) store_as<__half>(a.out, idx, z[k], wide);
            else store_as<__nv_bfloat16>(a.out, idx, z[k], wide);
        } else {
            // lanes 2 j, 2 j + 1 share a 16-element block, lanes 8 j .. 8 j + 7 a tiled 4-scale word
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(z[k][i]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            const uint32_t s = f32_to_e4m3(__fmul_rn(__fdiv_rn(amax, 6.0f), gs));
            const float sd = e4m3_to_f32(s);
            const uint32_t q = scale_to_e2m1x8(z[k], sd == 0.0f ? 0.0f : __fdiv_rn(gs, sd));
            if (a.sf_tiled) {                        // H % 64 == 0: words are whole
                const uint32_t two = s | __shfl_down_sync(0xffffffffu, s, 2) << 8;
                const uint32_t four = two | __shfl_down_sync(0xffffffffu, two, 4) << 16;
                if (in[k] && (c & 7) == 0)
                    *reinterpret_cast<uint32_t*>(a.sf + ((row >> 7) * (a.H >> 6) + (c >> 3)) * 512 + (row & 31) * 16 +
                                                 ((row >> 5) & 3) * 4) = four;
            } else if (in[k] && (c & 1) == 0) {
                a.sf[row * (a.H >> 4) + (c >> 1)] = static_cast<uint8_t>(s);
            }
            if (in[k]) *reinterpret_cast<uint32_t*>(a.q + row * (a.H >> 1) + 4 * c) = q;
        }
    }
}

template <typename T, int TPR, int V>
cudaError_t launch(const NormLaunch& a, cudaStream_t stream)
{
    // rows of a warp or less: four warps to a block once that still leaves every SM a block
    const int threads = TPR > 32 ? TPR : a.rows * TPR >= 32 * 1024 ? 128 : 32;
    const int64_t per_block = TPR > 32 ? 1 : threads / TPR;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>((a.rows + per_block - 1) / per_block), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return a.q ? cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, TPR, V, true>, a)
               : cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, TPR, V, false>, a);
}

template <typename T, int TPR>
cudaError_t launch_v(const NormLaunch& a, cudaStream_t stream)
{
    if constexpr (TPR < 32) {
        return launch<T, TPR, 1>(a, stream);
    } else {
        switch ((a.H / 8 + TPR - 1) / TPR) {
            case 1: return launch<T, TPR, 1>(a, stream);
            case 2: return launch<T, TPR, 2>(a, stream);
            case 3: return launch<T, TPR, 3>(a, stream);
            case 4: return launch<T, TPR, 4>(a, stream);
            default: return cudaErrorInvalidValue;
        }
    }
}

template <typename T>
cudaError_t launch_t(const NormLaunch& a, cudaStream_t stream, int num_sms)
{
    // Threads per row: as few as hold the row in four vectors each (16384 x 6144 bf16 with post_weight
    // and gate on 256 threads 139 us, on 512 160), two of fp32 (16384 x 8192 on 512 threads 315 us,
    // on 256 344); with no more rows than SMs the row is spread wider, one vector per thread. (The
    // threads of a row set the order of its sums: batches on the two sides may differ in last bits.)
    const int64_t v = a.rows <= num_sms ? 1 : sizeof(T) == 4 ? 2 : 4;
    if (a.H <= 64) return launch_v<T, 8>(a, stream);
    if (a.H <= 128) return launch_v<T, 16>(a, stream);
    if (a.H <= 256 * v) return launch_v<T, 32>(a, stream);
    if (a.H <= 2048 * v) return launch_v<T, 256>(a, stream);
    if (a.H <= 4096 * v) return launch_v<T, 512>(a, stream);
    return launch_v<T, 1024>(a, stream);
}

}  // namespace

cudaError_t launch_residual_norm(const NormLaunch& args, cudaStream_t stream, int num_sms)
{
    // every fp32 access 32-byte aligned: the weights, and the rows of fp32 tensors
    NormLaunch a = args;
    uintptr_t all = reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.b) |
                    reinterpret_cast<uintptr_t>(a.post) | reinterpret_cast<uintptr_t>(a.gate);
    if (a.dtype == 2)
        all |= reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.r) |
               static_cast<uintptr_t>(a.ld_x * 4) | static_cast<uintptr_t>(a.y ? a.ld_y * 4 : 0) |
               static_cast<uintptr_t>(a.r ? a.ld_r * 4 : 0);
    if (!a.q && a.out_dt == 2) all |= reinterpret_cast<uintptr_t>(a.out);
    a.wide = (all & 31u) == 0 ? 1 : 0;
    switch (a.dtype) {
        case 0: return launch_t<__nv_bfloat16>(a, stream, num_sms);
        case 1: return launch_t<__half>(a, stream, num_sms);
        case 2: return launch_t<float>(a, stream, num_sms);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace nvfp4
