// Global gradient norm over many tensors, and clipping by it.
//
//   norm  = sqrt(sum over all elements of g^2)
//   scale = max_norm / norm where norm is finite and above max_norm, else 1
//   out   = RN(g * scale), each element rounded once to its tensor's type
//
// The tensors are cut into chunks of 16384 elements counted from each one's
// first; a chunk's squares are summed in fp32 by a fixed order that does not
// depend on its alignment, the chunks' sums in fp64 in a fixed order.
#include "rlk_train.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;

// the tensor of a launch that holds its chunk c
__device__ __forceinline__ int tensor_of(const ClipTable& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <int kType>
__device__ __forceinline__ float load_as_float(const void* p, int64_t i) {
    if constexpr (kType == RLK_DTYPE_F32) return static_cast<const float*>(p)[i];
    else if constexpr (kType == RLK_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    else return __half2float(static_cast<const __half*>(p)[i]);
}

template <int kType>
__device__ __forceinline__ void store_from_float(void* p, int64_t i, float v) {
    if constexpr (kType == RLK_DTYPE_F32) static_cast<float*>(p)[i] = v;
    else if constexpr (kType == RLK_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

template <int kType>
__device__ __forceinline__ float chunk_sumsq(const void* p, int64_t b, int64_t e) {
    float s = 0.0f;
    for (int64_t i = b + threadIdx.x; i < e; i += kThreads) {
        const float v = load_as_float<kType>(p, i);
        s = __fmaf_rn(v, v, s);
    }
    return s;
}

__global__ void __launch_bounds__(kThreads) k_grad_sumsq(const __grid_constant__ ClipTable t,
                                                         float* partials) {
    __shared__ float smem[kThreads / 32];
    const int total = t.first[t.count];
    for (int c = blockIdx.x; c < total; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int64_t b = static_cast<int64_t>(c - t.first[k]) * kClipChunk;
        const int64_t e = b + kClipChunk < t.e[k].n ? b + kClipChunk : t.e[k].n;
        float s = t.dtype[k] == RLK_DTYPE_F32    ? chunk_sumsq<RLK_DTYPE_F32>(t.e[k].in, b, e)
                  : t.dtype[k] == RLK_DTYPE_BF16 ? chunk_sumsq<RLK_DTYPE_BF16>(t.e[k].in, b, e)
                                                 : chunk_sumsq<RLK_DTYPE_F16>(t.e[k].in, b, e);
        s = warp_sum(s);
        if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kThreads / 32; ++i) s = __fadd_rn(s, smem[i]);
            partials[c] = s;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(1024) k_grad_norm_final(const float* partials, int64_t n,
                                                          double max_norm, float* out_norm,
                                                          float* out_scale, int32_t* status) {
    __shared__ double smem[32];
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 1024) v += static_cast<double>(partials[i]);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = warp_sum(smem[threadIdx.x]);
        if (threadIdx.x == 0) {
            const double norm = sqrt(v);
            const bool finite = norm < static_cast<double>(CUDART_INF_F);
            if (out_norm) *out_norm = static_cast<float>(norm);
            if (out_scale) *out_scale = finite && norm > max_norm ? static_cast<float>(max_norm / norm) : 1.0f;
            if (!finite) report_status(status, RLK_ERR_NONFINITE);
        }
    }
}

template <int kType>
__device__ __forceinline__ void chunk_scale(const ClipEntry& t, int64_t b, int64_t e, float scale) {
    for (int64_t i = b + threadIdx.x; i < e; i += kThreads)
        store_from_float<kType>(t.out, i, __fmul_rn(load_as_float<kType>(t.in, i), scale));
}

__global__ void __launch_bounds__(kThreads) k_grad_scale(const __grid_constant__ ClipTable t,
                                                         const float* scale_ptr) {
    const float scale = *scale_ptr;
    const int total = t.first[t.count];
    for (int c = blockIdx.x; c < total; c += gridDim.x) {
        const int k = tensor_of(t, c);
        if (scale == 1.0f && t.e[k].in == t.e[k].out) continue;
        const int64_t b = static_cast<int64_t>(c - t.first[k]) * kClipChunk;
        const int64_t e = b + kClipChunk < t.e[k].n ? b + kClipChunk : t.e[k].n;
        if (t.dtype[k] == RLK_DTYPE_F32) chunk_scale<RLK_DTYPE_F32>(t.e[k], b, e, scale);
        else if (t.dtype[k] == RLK_DTYPE_BF16) chunk_scale<RLK_DTYPE_BF16>(t.e[k], b, e, scale);
        else chunk_scale<RLK_DTYPE_F16>(t.e[k], b, e, scale);
    }
}

int blocks_for(const ClipTable& t) {
    const int total = t.first[t.count];
    return total < 152 * 8 ? total : 152 * 8;
}

}  // namespace

cudaError_t launch_grad_sumsq(const ClipTable& t, float* partials, cudaStream_t stream) {
    k_grad_sumsq<<<blocks_for(t), kThreads, 0, stream>>>(t, partials);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm_final(const float* partials, int64_t n, double max_norm,
                                   float* out_norm, float* out_scale, int32_t* status,
                                   cudaStream_t stream) {
    k_grad_norm_final<<<1, 1024, 0, stream>>>(partials, n, max_norm, out_norm, out_scale, status);
    return cudaGetLastError();
}

cudaError_t launch_grad_scale(const ClipTable& t, const float* scale, cudaStream_t stream) {
    k_grad_scale<<<blocks_for(t), kThreads, 0, stream>>>(t, scale);
    return cudaGetLastError();
}

}  // namespace rlk
