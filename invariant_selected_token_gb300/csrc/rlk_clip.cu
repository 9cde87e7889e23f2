// Global gradient norm over many tensors, and clipping by it.
//
//   norm  = sqrt(sum over all elements of g^2)
//   scale = max_norm / norm where norm is finite and above max_norm, else 1
//   out   = RN(g * scale), each element rounded once to its tensor's type
//
// Order of the sum, which depends on the tensors' sizes alone: a tensor is cut
// into chunks of 2048 elements counted from its first, a warp's work each.
// With E elements in 16 bytes, class i mod 32 E of a chunk's elements is
// summed ascending in fp32, the classes by a fixed tree in fp32; chunk c of a
// launch goes to warp c mod (912 * 8) in ascending order, and the warps' sums
// are added by a fixed tree, these last two as pairs of floats.  An element's
// class does not depend on its address: 16-byte loads take whole aligned
// vectors wherever the tensor starts, and the lane that has a vector owns its
// elements' classes; only where the classes then lie in the lane's registers
// changes, and an exchange through shared memory undoes that.
//
// Sets of at most kClipClusterChunks chunks in at most 64 tensors run as one
// cluster of 8 CTAs in one launch: sums, norm and scaling.  Larger ones take a
// launch for the sums and one for the scaling, whose CTAs each form the norm
// from the at most 912 CTAs' sums; the second walks the chunks backwards, from
// those that the first left in L2.  No CTA-wide barrier stands between a
// warp's loads: chunks of 16384 elements by a whole CTA, with two barriers
// each, reached 5.6 TB/s where warps alone reach %SUMSQ%.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kClipCluster = 8;

template <int kType>
struct Elem;
template <>
struct Elem<RLK_DTYPE_F32> {
    using T = float;
    static constexpr int kPer = 4;  // in 16 bytes
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
};
template <>
struct Elem<RLK_DTYPE_BF16> {
    using T = __nv_bfloat16;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<RLK_DTYPE_F16> {
    using T = __half;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float get(T v) { return __half2float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};

template <int kType>
union Vec {
    uint4 raw;
    typename Elem<kType>::T e[Elem<kType>::kPer];
    __device__ Vec() {}
};

// Elements [s, s + kPer) of p[0 .. len), 16-byte aligned; those outside are zero.
template <int kType>
__device__ __forceinline__ void load_vec(Vec<kType>& v, const typename Elem<kType>::T* p, int s, int len) {
    constexpr int E = Elem<kType>::kPer;
    if (s >= 0 && s + E <= len) {
        v.raw = *reinterpret_cast<const uint4*>(p + s);
    } else {
        v.raw = make_uint4(0u, 0u, 0u, 0u);
        if (s < len) {
#pragma unroll
            for (int r = 0; r < E; ++r)
                if (s + r >= 0 && s + r < len) v.e[r] = p[s + r];
        }
    }
}

// How many elements before p the 16-byte line starts in which p lies.
template <int kType>
__device__ __forceinline__ int lead_of(const typename Elem<kType>::T* p) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(*p));
}

// Sum of squares of one chunk p[0 .. len) by a warp, on every lane.
template <int kType>
__device__ __forceinline__ float chunk_sumsq(const void* base, int64_t at, int len, float* exchange) {
    using El = Elem<kType>;
    constexpr int E = El::kPer, kBatch = 4, kStep = 32 * E;
    const int lane = threadIdx.x & 31;
    const typename El::T* p = static_cast<const typename El::T*>(base) + at;
    const int lead = lead_of<kType>(p);
    float acc[E] = {};
    for (int s0 = lane * E - lead; s0 < len; s0 += kBatch * kStep) {
        Vec<kType> v[kBatch];
#pragma unroll
        for (int m = 0; m < kBatch; ++m) load_vec<kType>(v[m], p, s0 + m * kStep, len);
#pragma unroll
        for (int m = 0; m < kBatch; ++m) {
#pragma unroll
            for (int r = 0; r < E; ++r) {
                const float x = El::get(v[m].e[r]);
                acc[r] = __fmaf_rn(x, x, acc[r]);
            }
        }
    }
    if (lead != 0) {
        __syncwarp();
#pragma unroll
        for (int r = 0; r < E; ++r) exchange[(lane * E + r - lead + kStep) % kStep] = acc[r];
        __syncwarp();
#pragma unroll
        for (int r = 0; r < E; ++r) acc[r] = exchange[lane * E + r];
    }
#pragma unroll
    for (int n = E / 2; n >= 1; n >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) acc[i] = __fadd_rn(acc[2 * i], acc[2 * i + 1]);
    }
    return warp_sum(acc[0]);
}

template <int kType>
__device__ __forceinline__ void chunk_scale(const ClipEntry& t, int64_t at, int len, float scale) {
    using El = Elem<kType>;
    constexpr int E = El::kPer, kBatch = 4, kStep = 32 * E;
    const int lane = threadIdx.x & 31;
    const typename El::T* p = static_cast<const typename El::T*>(t.in) + at;
    typename El::T* o = static_cast<typename El::T*>(t.out) + at;
    const int lead = lead_of<kType>(p);
    if (lead == lead_of<kType>(o)) {
        for (int s0 = lane * E - lead; s0 < len; s0 += kBatch * kStep) {
            Vec<kType> v[kBatch];
#pragma unroll
            for (int m = 0; m < kBatch; ++m) load_vec<kType>(v[m], p, s0 + m * kStep, len);
#pragma unroll
            for (int m = 0; m < kBatch; ++m) {
                const int s = s0 + m * kStep;
#pragma unroll
                for (int r = 0; r < E; ++r) v[m].e[r] = El::put(__fmul_rn(El::get(v[m].e[r]), scale));
                if (s >= 0 && s + E <= len) {
                    __stcs(reinterpret_cast<uint4*>(o + s), v[m].raw);
                } else if (s < len) {
#pragma unroll
                    for (int r = 0; r < E; ++r)
                        if (s + r >= 0 && s + r < len) o[s + r] = v[m].e[r];
                }
            }
        }
    } else {
        // input and output lie differently in their 16 bytes: element by element
#pragma unroll 8
        for (int i = lane; i < len; i += 32) o[i] = El::put(__fmul_rn(El::get(p[i]), scale));
    }
}

// The tensor that holds chunk c; `near`, the one that held this warp's last chunk, is tried first.
template <typename Table>
__device__ __forceinline__ int tensor_of(const Table& t, int c, int near) {
    if (t.first[near] <= c && c < t.first[near + 1]) return near;
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <typename Table>
__device__ __forceinline__ float table_sumsq(const Table& t, int c, int& near, float* exchange) {
    const int k = near = tensor_of(t, c, near);
    const int64_t at = static_cast<int64_t>(c - t.first[k]) * kClipChunk, left = t.e[k].n - at;
    const int len = left < kClipChunk ? static_cast<int>(left) : kClipChunk;
    return t.dtype[k] == RLK_DTYPE_F32    ? chunk_sumsq<RLK_DTYPE_F32>(t.e[k].in, at, len, exchange)
           : t.dtype[k] == RLK_DTYPE_BF16 ? chunk_sumsq<RLK_DTYPE_BF16>(t.e[k].in, at, len, exchange)
                                          : chunk_sumsq<RLK_DTYPE_F16>(t.e[k].in, at, len, exchange);
}

template <typename Table>
__device__ __forceinline__ void table_scale(const Table& t, int c, int& near, float scale) {
    const int k = near = tensor_of(t, c, near);
    if (scale == 1.0f && t.e[k].in == t.e[k].out) return;
    const int64_t at = static_cast<int64_t>(c - t.first[k]) * kClipChunk, left = t.e[k].n - at;
    const int len = left < kClipChunk ? static_cast<int>(left) : kClipChunk;
    if (t.dtype[k] == RLK_DTYPE_F32) chunk_scale<RLK_DTYPE_F32>(t.e[k], at, len, scale);
    else if (t.dtype[k] == RLK_DTYPE_BF16) chunk_scale<RLK_DTYPE_BF16>(t.e[k], at, len, scale);
    else chunk_scale<RLK_DTYPE_F16>(t.e[k], at, len, scale);
}

// A CTA's sum from its 8 warps', on thread 0.
__device__ __forceinline__ float2 warps_sum(float2 v, float2* smem) {
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kWarps; ++i) v = pair_add(v, smem[i]);
    }
    return v;
}

// The slots' sum by a CTA of 256 threads, and from it (norm, scale); every thread gets them.
__device__ __forceinline__ float2 norm_and_scale(const float2* slots, int n, double max_norm, float2* smem) {
    __shared__ float2 result;
    float2 v = pair_of(0.0f);
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) v = pair_add(v, slots[i]);
    v = warps_sum(warp_sum(v), smem);
    if (threadIdx.x == 0) {
        const float norm = __fsqrt_rn(__fadd_rn(v.x, v.y));
        const bool shrink = norm < CUDART_INF_F && static_cast<double>(norm) > max_norm;
        result = make_float2(norm, shrink ? __fdiv_rn(static_cast<float>(max_norm), norm) : 1.0f);
    }
    __syncthreads();
    return result;
}

__device__ __forceinline__ void write_norm(const ClipOut& o, float2 r) {
    *o.norm = r.x;
    if (o.scale) *o.scale = r.y;
    if (!(r.x < CUDART_INF_F)) report_status(o.status, RLK_ERR_NONFINITE);
}

// ---------------------------------------------------------------- one launch
// CTA r of the cluster stands for CTAs r, r + 8, ... of the launch for sums: its warps take those
// CTAs' chunks, at most one each, so the sums meet in the same order.
__global__ void __launch_bounds__(kThreads) k_clip_cluster(const __grid_constant__ ClipTableSmall t,
                                                           const ClipOut o) {
    __shared__ float exchange[kWarps][32 * 8];
    __shared__ float2 chunks[kClipClusterChunks];  // every chunk's sum, in every CTA
    __shared__ float2 slots[kClipClusterChunks / kWarps];
    __shared__ float2 tmp[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int total = t.first[t.count];
    int near = 0;
    bool started = false;
    for (int c = warp * kClipCluster + rank; c < total; c += kClipCluster * kWarps) {
        const float s = table_sumsq(t, c, near, exchange[warp]);
        if (!started) cluster.barrier_wait();  // every CTA has started: its shared memory may be written
        started = true;
        if (lane < kClipCluster) cluster.map_shared_rank(chunks, lane)[c] = pair_of(s);
    }
    if (!started) cluster.barrier_wait();
    cluster.sync();
    const int n = (total + kWarps - 1) / kWarps;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        float2 v = chunks[i * kWarps];
        for (int k = i * kWarps + 1; k < total && k < (i + 1) * kWarps; ++k) v = pair_add(v, chunks[k]);
        slots[i] = v;
    }
    __syncthreads();
    const float2 r = norm_and_scale(slots, n, o.max_norm, tmp);
    if (rank == 0 && threadIdx.x == 0) write_norm(o, r);
    if (!o.scale) return;
    for (int c = warp * kClipCluster + rank; c < total; c += kClipCluster * kWarps) table_scale(t, c, near, r.y);
}

// ---------------------------------------------------------------- two launches
__global__ void __launch_bounds__(kThreads, 6) k_grad_sumsq(const __grid_constant__ ClipTable t, float2* slots) {
    __shared__ float exchange[kWarps][32 * 8];
    __shared__ float2 tmp[kWarps];
    ptx::grid_dependents_launch();
    const int total = t.first[t.count], warp = threadIdx.x >> 5;
    float2 sum = pair_of(0.0f);
    int near = 0;
    for (int c = blockIdx.x * kWarps + warp; c < total; c += kClipSlots * kWarps)
        sum = pair_add(sum, pair_of(table_sumsq(t, c, near, exchange[warp])));
    sum = warps_sum(sum, tmp);
    if (threadIdx.x == 0) slots[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const float2* slots, int n, const ClipOut o) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o.max_norm, tmp);
    if (threadIdx.x == 0) write_norm(o, r);
}

__global__ void __launch_bounds__(kThreads, 6) k_grad_scale(const __grid_constant__ ClipTable t, const float2* slots,
                                                         int n, const ClipOut o, int write) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o.max_norm, tmp);
    const float scale = r.y;
    if (write && blockIdx.x == 0 && threadIdx.x == 0) write_norm(o, r);
    int near = 0;
    for (int c = t.first[t.count] - 1 - static_cast<int>(blockIdx.x * kWarps + (threadIdx.x >> 5)); c >= 0;
         c -= static_cast<int>(gridDim.x) * kWarps)
        table_scale(t, c, near, scale);
}

template <typename... Args>
cudaError_t launch_after(void (*kernel)(Args...), int blocks, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_clip_cluster(const ClipTableSmall& t, const ClipOut& o, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(kClipCluster, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kClipCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_clip_cluster, t, o);
}

cudaError_t launch_grad_sumsq(const ClipTable& t, float2* slots, cudaStream_t stream) {
    k_grad_sumsq<<<clip_launch_slots(t.first[t.count]), kThreads, 0, stream>>>(t, slots);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm(const float2* slots, int n, const ClipOut& o, cudaStream_t stream) {
    return launch_after(k_grad_norm, 1, stream, slots, n, o);
}

cudaError_t launch_grad_scale(const ClipTable& t, const float2* slots, int n, const ClipOut& o, bool write,
                              cudaStream_t stream) {
    return launch_after(k_grad_scale, clip_launch_slots(t.first[t.count]), stream, t, slots, n, o, int(write));
}

}  // namespace rlk
