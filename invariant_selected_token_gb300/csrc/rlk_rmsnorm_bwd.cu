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
// summed over at most 304 (152 for rows wider than 4096) ranges of consecutive
// rows, one CTA each, then over the ranges, in an order that T and H fix.
#include "rlk_contract.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

constexpr int cta_threads(int kWarps) { return kWarps == 32 ? 1024 : 512; }

template <int kType>
struct Raw8 {  // 8 features as loaded
    uint4 w[kType == RLK_DTYPE_F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const char* p = static_cast<const char*>(base) + i * (kType == RLK_DTYPE_F32 ? 4 : 2);
#pragma unroll
        for (int k = 0; k < (kType == RLK_DTYPE_F32 ? 2 : 1); ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < (kType == RLK_DTYPE_F32 ? 2 : 1); ++k) w[k] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ float at(int j) const {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(w);
        if constexpr (kType == RLK_DTYPE_F32) return __uint_as_float(q[j]);
        else return (j & 1) ? bf_hi(q[j / 2]) : bf_lo(q[j / 2]);
    }
};

// A team of kWarps warps (a power of two, one thread per 8 features) takes a row, a CTA's teams
// every kTeams-th row of its range.  The next row's x and grad_out are loaded before the current
// one is reduced, so that the reduction and its barrier hide behind them.
template <int kWarps, int kGo, int kGx>
__global__ void __launch_bounds__(cta_threads(kWarps), kWarps == 32 ? 1 : 2) k_rmsnorm_backward(const RmsBwdArgs a) {
    constexpr int kThreads = cta_threads(kWarps), kTeams = kThreads / 32 / kWarps;
    __shared__ float2 part[2][kThreads / 32];
    __shared__ __align__(16) float dg_teams[kTeams > 1 ? kThreads * 8 : 1];
    ptx::grid_dependents_launch();
    const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * kWarps);
    const int warp = (threadIdx.x >> 5) % kWarps;
    const int i0 = (warp * 32 + lane) * 8;
    const bool in = i0 < a.H;
    const int64_t r0 = static_cast<int64_t>(a.T) * blockIdx.x / gridDim.x;
    const int64_t r1 = static_cast<int64_t>(a.T) * (blockIdx.x + 1) / gridDim.x;
    const float inv_h_den = static_cast<float>(a.H);
    Raw8<RLK_DTYPE_BF16> gam, x, x_next;
    Raw8<kGo> dy, dy_next;
    Raw8<kGx> res;
    gam.clear();
    x_next.clear();
    dy_next.clear();
    res.clear();
    float dg[8] = {};
    int64_t t = r0 + team;
    if (in) {
        gam.load(a.gamma, i0);
        if (t < r1) {
            x_next.load(a.x, t * a.H + i0);
            dy_next.load(a.grad_out, t * a.H + i0);
        }
    }
    int slot = 0;
    for (; t < r1; t += kTeams) {
        x = x_next;
        dy = dy_next;
        if (in) {
            if (a.grad_res) res.load(a.grad_res, t * a.H + i0);
            if (t + kTeams < r1) {
                x_next.load(a.x, (t + kTeams) * a.H + i0);
                dy_next.load(a.grad_out, (t + kTeams) * a.H + i0);
            }
        }
        // the forward's tree: pairs of features, then lanes, then warps
        float s2[4], d = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            s2[k] = __fadd_rn(__fmul_rn(x.at(2 * k), x.at(2 * k)), __fmul_rn(x.at(2 * k + 1), x.at(2 * k + 1)));
        float s = __fadd_rn(__fadd_rn(s2[0], s2[1]), __fadd_rn(s2[2], s2[3]));
#pragma unroll
        for (int k = 0; k < 8; ++k) d = __fmaf_rn(__fmul_rn(dy.at(k), gam.at(k)), x.at(k), d);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
            d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
        }
        if constexpr (kWarps > 1) {
            if (lane == 0) part[slot][team * kWarps + warp] = make_float2(s, d);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kWarps) : "memory");
            const float2 p = part[slot][team * kWarps + lane % kWarps];
            s = p.x;
            d = p.y;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) {
                s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
                d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
            }
            slot ^= 1;  // a team's warps are never more than one row apart
        }
        const float rstd = contract_rsqrt(__fadd_rn(__fdiv_rn(s, inv_h_den), a.eps));
        const float c = __fdiv_rn(__fmul_rn(__fmul_rn(rstd, rstd), d), inv_h_den);
        if (in) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float up = __fmul_rn(dy.at(k), gam.at(k));
                o[k] = __fmaf_rn(rstd, __fmaf_rn(-x.at(k), c, up), res.at(k));
                dg[k] = __fmaf_rn(dy.at(k), __fmul_rn(x.at(k), rstd), dg[k]);
            }
            store8<kGx>(a.grad_x, t * a.H + i0, o);
        }
    }
    if (!a.grad_gamma) return;
    float* const out = a.parts + static_cast<int64_t>(blockIdx.x) * a.H;
    if constexpr (kTeams == 1) {
        if (in) store8<RLK_DTYPE_F32>(out, i0, dg);
    } else {
        // the teams' sums in ascending order
        store8<RLK_DTYPE_F32>(dg_teams, team * kWarps * 256 + i0, dg);
        __syncthreads();
        for (int i = threadIdx.x; i < a.H; i += kThreads) {
            float v = dg_teams[i];
#pragma unroll
            for (int k = 1; k < kTeams; ++k) v = __fadd_rn(v, dg_teams[k * kWarps * 256 + i]);
            out[i] = v;
        }
    }
}

// grad_gamma from the ranges' sums: 32 threads per feature, each taking every 32nd range in
// ascending order, then pairwise.
__global__ void __launch_bounds__(1024) k_rmsnorm_gamma_sum(const float* parts, int ranges, int H,
                                                            float* out) {
    __shared__ float smem[32][33];
    const int c = threadIdx.x & 31, row = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    ptx::grid_dependency_wait();
    float s = 0.0f;
#pragma unroll 5
    for (int r = row; r < ranges; r += 32) s = __fadd_rn(s, parts[static_cast<int64_t>(r) * H + col]);
    smem[row][c] = s;
    __syncthreads();
    s = warp_sum(smem[c][row]);  // feature `row` of the CTA's 32, one range class per lane
    if (c == 0) out[blockIdx.x * 32 + row] = s;
}

template <int kWarps>
void launch_row(const RmsBwdArgs& a, int blocks, cudaStream_t stream) {
    constexpr int kThreads = cta_threads(kWarps);
    if (a.go_dtype == RLK_DTYPE_F32) {
        if (a.gx_dtype == RLK_DTYPE_F32)
            k_rmsnorm_backward<kWarps, RLK_DTYPE_F32, RLK_DTYPE_F32><<<blocks, kThreads, 0, stream>>>(a);
        else
            k_rmsnorm_backward<kWarps, RLK_DTYPE_F32, RLK_DTYPE_BF16><<<blocks, kThreads, 0, stream>>>(a);
    } else {
        if (a.gx_dtype == RLK_DTYPE_F32)
            k_rmsnorm_backward<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_F32><<<blocks, kThreads, 0, stream>>>(a);
        else
            k_rmsnorm_backward<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_BF16><<<blocks, kThreads, 0, stream>>>(a);
    }
}

}  // namespace

cudaError_t launch_rmsnorm_backward(const RmsBwdArgs& a, cudaStream_t stream) {
    const int blocks = rmsnorm_backward_ranges(a.T, a.H);
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
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.grad_gamma) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(a.H / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rmsnorm_gamma_sum, static_cast<const float*>(a.parts), blocks, a.H, a.grad_gamma);
}

}  // namespace rlk
