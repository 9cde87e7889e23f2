// Backward of the strict RMSNorm.  Per row, with x the row that was
// normalised (after the residual addition), dy = grad_out and the forward's
// rstd (the same tree over the same squares, so the same bits):
//
//   up_i   = dy_i gamma_i
//   c      = rstd^2 / H * sum_i up_i x_i
//   grad_x = rstd (up_i - x_i c) + grad_residual_i
//   grad_gamma_i = sum over rows of dy_i x_i rstd
//
// A row's grad_x does not depend on the batch around it.  grad_gamma is
// summed over min(T, 304) ranges of consecutive rows, ascending in each, and
// the ranges' sums by a fixed order.
#include "rlk_contract.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int kType>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
    if constexpr (kType == RLK_DTYPE_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf_lo(w[k]);
            v[2 * k + 1] = bf_hi(w[k]);
        }
    }
}

template <int kType>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
    if constexpr (kType == RLK_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) |
                   (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One thread per 8 features; kWarps warps (a power of two) cover the row.
template <int kWarps, int kGo, int kGx>
__global__ void __launch_bounds__(kWarps * 32) k_rmsnorm_backward(const RmsBwdArgs a) {
    __shared__ float sq[kWarps], dot[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i0 = threadIdx.x * 8;
    const bool in = i0 < a.H;
    const int64_t r0 = static_cast<int64_t>(a.T) * blockIdx.x / gridDim.x;
    const int64_t r1 = static_cast<int64_t>(a.T) * (blockIdx.x + 1) / gridDim.x;
    float gam[8] = {}, dg[8] = {};
    if (in) load8<RLK_DTYPE_BF16>(a.gamma, i0, gam);
    for (int64_t t = r0; t < r1; ++t) {
        float x[8] = {}, dy[8] = {}, up[8];
        if (in) {
            load8<RLK_DTYPE_BF16>(a.x, t * a.H + i0, x);
            load8<kGo>(a.grad_out, t * a.H + i0, dy);
        }
        // the forward's tree: pairs of features, then lanes, then warps
        float s = __fadd_rn(__fadd_rn(__fadd_rn(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1])),
                                      __fadd_rn(__fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3]))),
                            __fadd_rn(__fadd_rn(__fmul_rn(x[4], x[4]), __fmul_rn(x[5], x[5])),
                                      __fadd_rn(__fmul_rn(x[6], x[6]), __fmul_rn(x[7], x[7]))));
        float d = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            up[k] = __fmul_rn(dy[k], gam[k]);
            d = __fmaf_rn(up[k], x[k], d);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
            d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
        }
        if (lane == 0) {
            sq[warp] = s;
            dot[warp] = d;
        }
        __syncthreads();
        float ps[kWarps], pd[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            ps[i] = sq[i];
            pd[i] = dot[i];
        }
#pragma unroll
        for (int n = kWarps / 2; n >= 1; n >>= 1) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                ps[i] = __fadd_rn(ps[2 * i], ps[2 * i + 1]);
                pd[i] = __fadd_rn(pd[2 * i], pd[2 * i + 1]);
            }
        }
        __syncthreads();
        const float rstd = contract_rsqrt(__fadd_rn(__fdiv_rn(ps[0], static_cast<float>(a.H)), a.eps));
        const float c = __fdiv_rn(__fmul_rn(__fmul_rn(rstd, rstd), pd[0]), static_cast<float>(a.H));
        if (in) {
            float o[8], res[8] = {};
            if (a.grad_res) load8<kGx>(a.grad_res, t * a.H + i0, res);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[k] = __fmaf_rn(rstd, __fmaf_rn(-x[k], c, up[k]), res[k]);
                dg[k] = __fmaf_rn(dy[k], __fmul_rn(x[k], rstd), dg[k]);
            }
            store8<kGx>(a.grad_x, t * a.H + i0, o);
        }
    }
    if (in && a.grad_gamma) store8<RLK_DTYPE_F32>(a.parts, static_cast<int64_t>(blockIdx.x) * a.H + i0, dg);
}

// grad_gamma from the ranges' sums: 8 threads per feature, each taking every
// 8th range in ascending order, then pairwise.
__global__ void __launch_bounds__(256) k_rmsnorm_gamma_sum(const float* parts, int ranges, int H,
                                                           float* out) {
    __shared__ float smem[8][32];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
    float s = 0.0f;
    for (int r = row; r < ranges; r += 8) s = __fadd_rn(s, parts[static_cast<int64_t>(r) * H + col]);
    smem[row][threadIdx.x & 31] = s;
    __syncthreads();
    if (row == 0) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = smem[i][threadIdx.x];
        out[col] = __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                             __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
    }
}

template <int kWarps>
void launch_row(const RmsBwdArgs& a, int blocks, cudaStream_t stream) {
    if (a.go_dtype == RLK_DTYPE_F32) {
        if (a.gx_dtype == RLK_DTYPE_F32)
            k_rmsnorm_backward<kWarps, RLK_DTYPE_F32, RLK_DTYPE_F32><<<blocks, kWarps * 32, 0, stream>>>(a);
        else
            k_rmsnorm_backward<kWarps, RLK_DTYPE_F32, RLK_DTYPE_BF16><<<blocks, kWarps * 32, 0, stream>>>(a);
    } else {
        if (a.gx_dtype == RLK_DTYPE_F32)
            k_rmsnorm_backward<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_F32><<<blocks, kWarps * 32, 0, stream>>>(a);
        else
            k_rmsnorm_backward<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_BF16><<<blocks, kWarps * 32, 0, stream>>>(a);
    }
}

}  // namespace

cudaError_t launch_rmsnorm_backward(const RmsBwdArgs& a, cudaStream_t stream) {
    const int blocks = a.T < kRmsBwdBlocks ? a.T : kRmsBwdBlocks;
    int warps = 1;
    while (warps * 256 < a.H) warps *= 2;
    if (blocks > 0) switch (warps) {
        case 1: launch_row<1>(a, blocks, stream); break;
        case 2: launch_row<2>(a, blocks, stream); break;
        case 4: launch_row<4>(a, blocks, stream); break;
        case 8: launch_row<8>(a, blocks, stream); break;
        case 16: launch_row<16>(a, blocks, stream); break;
        case 32: launch_row<32>(a, blocks, stream); break;
        default: return cudaErrorInvalidValue;
    }
    if (a.grad_gamma)
        k_rmsnorm_gamma_sum<<<a.H / 32, 256, 0, stream>>>(a.parts, blocks, a.H, a.grad_gamma);
    return cudaGetLastError();
}

}  // namespace rlk
