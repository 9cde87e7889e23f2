// The block norms' backward: the choice of the main kernel's instance, which
// go by the kind of the saved activations and grad_out's type, a translation
// unit each, and the launch that adds the ranges' sums up to the grad_gammas.
#include "rlk_block.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

// The grad_gammas from the ranges' sums: 32 threads per feature, each taking every 32nd range in
// ascending order, then pairwise.
__global__ void __launch_bounds__(1024)
    k_gamma_sums(const float* parts, int ranges, int H, float* grad_pre, float* grad_post) {
    __shared__ float smem[32][33];
    const int c = threadIdx.x & 31, row = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    ptx::grid_dependency_wait();
    float s = 0.0f;
#pragma unroll 5
    for (int r = row; r < ranges; r += 32) s = __fadd_rn(s, parts[static_cast<int64_t>(r) * 2 * H + col]);
    smem[row][c] = s;
    __syncthreads();
    s = warp_sum(smem[c][row]);  // feature `row` of the CTA's 32, one range class per lane
    const int at = blockIdx.x * 32 + row;
    if (c == 0 && at < H && grad_pre) grad_pre[at] = s;
    if (c == 0 && at >= H && grad_post) grad_post[at - H] = s;
}

}  // namespace

cudaError_t launch_block_bwd(const BlockBwdArgs& a, int format, cudaStream_t stream) {
    const int blocks = block_bwd_ranges(a.T);
    const bool f32 = a.go_dtype == RLK_DTYPE_F32;
    cudaError_t e = cudaSuccess;
    if (blocks > 0) switch (format) {
        case RLK_SAVED_BF16:
            e = f32 ? launch_block_bwd_bf16_f32(a, blocks, stream) : launch_block_bwd_bf16_bf16(a, blocks, stream);
            break;
        case RLK_SAVED_INT8:
            e = f32 ? launch_block_bwd_int8_f32(a, blocks, stream) : launch_block_bwd_int8_bf16(a, blocks, stream);
            break;
        default:
            e = f32 ? launch_block_bwd_e4m3_f32(a, blocks, stream) : launch_block_bwd_e4m3_bf16(a, blocks, stream);
    }
    if (e != cudaSuccess || (!a.grad_pre && !a.grad_post)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((a.grad_post ? 2 : 1) * a.H / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_gamma_sums, static_cast<const float*>(a.parts), blocks, a.H, a.grad_pre, a.grad_post);
}

}  // namespace rlk
