// Global gradient norm over many tensors, and clipping by it.
//
//   norm  = sqrt(sum over all elements of g^2)
//   scale = max_norm / norm where norm is finite and above max_norm, else 1
//   out   = RN(g * scale), each element rounded once to its tensor's type
//
// Order of the sum, which depends on the tensors' sizes alone: a tensor is cut
// into chunks of 16384 elements counted from its first.  With E elements in
// 16 bytes, class i mod 256 E of a chunk's elements is summed ascending in
// fp32, the classes by a fixed tree in fp32; chunk c of a launch goes to slot
// c mod 912 in ascending order and the slots are added by a fixed tree, both
// as pairs of floats.  An element's class does not depend on its address: 16-byte
// loads take whole aligned vectors wherever the tensor starts, and the thread
// that has a vector owns its elements' classes; only where the classes then
// lie in the thread's registers changes, and an exchange through shared
// memory undoes that.
//
// Sets of at most 48 chunks in at most 64 tensors run as one cluster of 8 CTAs in one launch: sums,
// norm and scaling.  Larger ones take a launch for the sums and one for the
// scaling, whose CTAs each form the norm from the at most 912 slots; the
// second walks the chunks backwards, from those that the first left in L2.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
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

struct ClipShared {
    float exchange[kThreads * 8];
    float warps[kThreads / 32];
};

// Sum of squares of one chunk p[0 .. len), by a group of 256 threads, on its thread 0.
template <int kType>
__device__ __forceinline__ float chunk_sumsq(const void* base, int64_t at, int len, ClipShared& sm) {
    using El = Elem<kType>;
    constexpr int E = El::kPer, kBatch = 4;
    const typename El::T* p = static_cast<const typename El::T*>(base) + at;
    const int lead = lead_of<kType>(p);
    float acc[E] = {};
    for (int s0 = static_cast<int>(threadIdx.x) * E - lead; s0 < len; s0 += kBatch * kThreads * E) {
        Vec<kType> v[kBatch];
#pragma unroll
        for (int m = 0; m < kBatch; ++m) load_vec<kType>(v[m], p, s0 + m * kThreads * E, len);
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
#pragma unroll
        for (int r = 0; r < E; ++r)
            sm.exchange[(static_cast<int>(threadIdx.x) * E + r - lead + kThreads * E) % (kThreads * E)] = acc[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < E; ++r) acc[r] = sm.exchange[threadIdx.x * E + r];
    }
#pragma unroll
    for (int n = E / 2; n >= 1; n >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) acc[i] = __fadd_rn(acc[2 * i], acc[2 * i + 1]);
    }
    const float s = warp_sum(acc[0]);
    if ((threadIdx.x & 31) == 0) sm.warps[threadIdx.x >> 5] = s;
    __syncthreads();
    float total = 0.0f;
    if (threadIdx.x == 0) {
        float w[kThreads / 32];
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) w[i] = sm.warps[i];
        total = __fadd_rn(__fadd_rn(__fadd_rn(w[0], w[1]), __fadd_rn(w[2], w[3])),
                          __fadd_rn(__fadd_rn(w[4], w[5]), __fadd_rn(w[6], w[7])));
    }
    __syncthreads();
    return total;
}

template <int kType>
__device__ __forceinline__ void chunk_scale(const ClipEntry& t, int64_t at, int len, float scale) {
    using El = Elem<kType>;
    constexpr int E = El::kPer, kBatch = 4;
    const typename El::T* p = static_cast<const typename El::T*>(t.in) + at;
    typename El::T* o = static_cast<typename El::T*>(t.out) + at;
    const int lead = lead_of<kType>(p);
    if (lead == lead_of<kType>(o)) {
        for (int s0 = static_cast<int>(threadIdx.x) * E - lead; s0 < len; s0 += kBatch * kThreads * E) {
            Vec<kType> v[kBatch];
#pragma unroll
            for (int m = 0; m < kBatch; ++m) load_vec<kType>(v[m], p, s0 + m * kThreads * E, len);
#pragma unroll
            for (int m = 0; m < kBatch; ++m) {
                const int s = s0 + m * kThreads * E;
                if (s >= len) break;
#pragma unroll
                for (int r = 0; r < E; ++r) v[m].e[r] = El::put(__fmul_rn(El::get(v[m].e[r]), scale));
                if (s >= 0 && s + E <= len) {
                    __stcs(reinterpret_cast<uint4*>(o + s), v[m].raw);
                } else {
#pragma unroll
                    for (int r = 0; r < E; ++r)
                        if (s + r >= 0 && s + r < len) o[s + r] = v[m].e[r];
                }
            }
        }
    } else {
        // input and output lie differently in their 16 bytes: element by element
#pragma unroll 8
        for (int i = threadIdx.x; i < len; i += kThreads) o[i] = El::put(__fmul_rn(El::get(p[i]), scale));
    }
}

// the tensor that holds chunk c
template <typename Table>
__device__ __forceinline__ int tensor_of(const Table& t, int c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
}

template <typename Table>
__device__ __forceinline__ float table_sumsq(const Table& t, int c, ClipShared& sm) {
    const int k = tensor_of(t, c);
    const int64_t at = static_cast<int64_t>(c - t.first[k]) * kClipChunk, left = t.e[k].n - at;
    const int len = left < kClipChunk ? static_cast<int>(left) : kClipChunk;
    return t.dtype[k] == RLK_DTYPE_F32    ? chunk_sumsq<RLK_DTYPE_F32>(t.e[k].in, at, len, sm)
           : t.dtype[k] == RLK_DTYPE_BF16 ? chunk_sumsq<RLK_DTYPE_BF16>(t.e[k].in, at, len, sm)
                                          : chunk_sumsq<RLK_DTYPE_F16>(t.e[k].in, at, len, sm);
}

template <typename Table>
__device__ __forceinline__ void table_scale(const Table& t, int c, float scale) {
    const int k = tensor_of(t, c);
    if (scale == 1.0f && t.e[k].in == t.e[k].out) return;
    const int64_t at = static_cast<int64_t>(c - t.first[k]) * kClipChunk, left = t.e[k].n - at;
    const int len = left < kClipChunk ? static_cast<int>(left) : kClipChunk;
    if (t.dtype[k] == RLK_DTYPE_F32) chunk_scale<RLK_DTYPE_F32>(t.e[k], at, len, scale);
    else if (t.dtype[k] == RLK_DTYPE_BF16) chunk_scale<RLK_DTYPE_BF16>(t.e[k], at, len, scale);
    else chunk_scale<RLK_DTYPE_F16>(t.e[k], at, len, scale);
}

// The slots' sum by a CTA of 256 threads, and from it (norm, scale); every thread gets them.
__device__ __forceinline__ float2 norm_and_scale(const float2* slots, int n, double max_norm, float2* smem) {
    __shared__ float2 result;
    float2 v = pair_of(0.0f);
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) v = pair_add(v, slots[i]);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 32; ++i) v = pair_add(v, smem[i]);
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
__global__ void __launch_bounds__(kThreads) k_clip_cluster(const __grid_constant__ ClipTableSmall t,
                                                           const ClipOut o) {
    __shared__ ClipShared sm;
    __shared__ float2 slots[kClipClusterChunks];
    __shared__ float2 tmp[kThreads / 32];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank());
    const int total = t.first[t.count];
    bool started = false;
    for (int c = rank; c < total; c += kClipCluster) {
        const float2 s = pair_of(table_sumsq(t, c, sm));
        if (!started) cluster.barrier_wait();  // every CTA has started: its shared memory may be written
        started = true;
        if (threadIdx.x == 0) {
            for (int r = 0; r < kClipCluster; ++r) cluster.map_shared_rank(slots, r)[c] = s;
        }
    }
    if (!started) cluster.barrier_wait();
    cluster.sync();
    const float2 r = norm_and_scale(slots, total, o.max_norm, tmp);
    if (rank == 0 && threadIdx.x == 0) write_norm(o, r);
    if (!o.scale) return;
    for (int c = rank; c < total; c += kClipCluster) table_scale(t, c, r.y);
}

// ---------------------------------------------------------------- two launches
__global__ void __launch_bounds__(kThreads) k_grad_sumsq(const __grid_constant__ ClipTable t, float2* slots) {
    __shared__ ClipShared sm;
    ptx::grid_dependents_launch();
    const int total = t.first[t.count];
    float2 sum = pair_of(0.0f);
    for (int c = blockIdx.x; c < total; c += kClipSlots) {
        const float s = table_sumsq(t, c, sm);
        if (threadIdx.x == 0) sum = pair_add(sum, pair_of(s));
    }
    if (threadIdx.x == 0) slots[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const float2* slots, int n, const ClipOut o) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o.max_norm, tmp);
    if (threadIdx.x == 0) write_norm(o, r);
}

__global__ void __launch_bounds__(kThreads) k_grad_scale(const __grid_constant__ ClipTable t, const float2* slots,
                                                         int n, const ClipOut o, int write) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o.max_norm, tmp);
    const float scale = r.y;
    if (write && blockIdx.x == 0 && threadIdx.x == 0) write_norm(o, r);
    for (int c = t.first[t.count] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) table_scale(t, c, scale);
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
    const int total = t.first[t.count];
    k_grad_sumsq<<<total < kClipSlots ? total : kClipSlots, kThreads, 0, stream>>>(t, slots);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm(const float2* slots, int n, const ClipOut& o, cudaStream_t stream) {
    return launch_after(k_grad_norm, 1, stream, slots, n, o);
}

cudaError_t launch_grad_scale(const ClipTable& t, const float2* slots, int n, const ClipOut& o, bool write,
                              cudaStream_t stream) {
    const int total = t.first[t.count];
    return launch_after(k_grad_scale, total < kClipSlots ? total : kClipSlots, stream, t, slots, n, o, int(write));
}

}  // namespace rlk
