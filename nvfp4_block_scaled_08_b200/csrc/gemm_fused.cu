// gemm_fused.cu -- the dense NVFP4 product with a fused epilogue: bias, activation and residual,
// the gated feed-forward product (16- or 32-bit or NVFP4 output) and its gradients. The
// kernel of the plain product (gemm.cu) on its few-token tiles, on 128 x 128 tiles and on CTA pairs
// (256 x 128, 256 x 256; no single-CTA tiles wider than 128), with a planner of its own (plan_fused);
// tiled scales only.
#include "gemm_epilogue.cuh"
#include "gemm_launch.cuh"

namespace nvfp4 {

template <int EPI>
static cudaError_t launch_epi(const GemmPlan& plan, const GemmLaunch& L, cudaStream_t stream, bool* encode_failed)
{
    if (plan.swap) {
        switch (plan.bn) {
            case 16: return run<16, true, false, true, false, false, false, false, EPI>(plan, L, stream, encode_failed);
            case 32: return run<32, true, false, true, false, false, false, false, EPI>(plan, L, stream, encode_failed);
            case 64: return run<64, true, false, true, false, false, false, false, EPI>(plan, L, stream, encode_failed);
            default: return cudaErrorInvalidValue;
        }
    }
    if (plan.pair && plan.bn == 256)
        return run<256, false, false, true, false, false, true, false, EPI>(plan, L, stream, encode_failed);
    if (plan.pair && plan.bn == 128)
        return run<128, false, false, true, false, false, true, false, EPI>(plan, L, stream, encode_failed);
    if (plan.bn == 128) return run<128, false, false, true, false, false, false, false, EPI>(plan, L, stream, encode_failed);
    return cudaErrorInvalidValue;
}

cudaError_t launch_gemm_fused(const GemmPlan& plan, const GemmLaunch& L, int epilogue, cudaStream_t stream,
                              bool* encode_failed)
{
    *encode_failed = false;
    if (plan.grid <= 0) return cudaSuccess;
    if (plan.groups != 1 || (plan.swap && plan.q_tiles != 1)) return cudaErrorInvalidValue;
    switch (epilogue) {
        case kEpiLinear: return launch_epi<kEpiLinear>(plan, L, stream, encode_failed);
        case kEpiGlu: return launch_epi<kEpiGlu>(plan, L, stream, encode_failed);
        case kEpiGluQuant: return launch_epi<kEpiGluQuant>(plan, L, stream, encode_failed);
        case kEpiGluGrad: return launch_epi<kEpiGluGrad>(plan, L, stream, encode_failed);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace nvfp4
