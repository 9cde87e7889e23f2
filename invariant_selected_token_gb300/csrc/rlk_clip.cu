// Global gradient norm over many tensors, and clipping by it.
//
//   norm  = sqrt(sum over all elements of g^2)
//   scale = max_norm / norm where norm is finite and above max_norm, else 1
//   out   = RN(g * scale), each element rounded once to its tensor's type
//
// Each tensor is cut into pieces of 16 KB, counted from the 16-byte line in
// which it starts; CTA c takes pieces c, c + CTAs, ... of all tensors, a
// thread the same four 16-byte vectors of each.  It loads its next piece's
// vectors before it works on the current one's, whatever tensor and type they
// belong to, and nothing but the end of the kernel needs a barrier.  A thread
// keeps one fp32 sum per place in its vectors (emptied into a second one every
// 16 pieces); a fixed tree adds them at the end, and the CTAs' sums are added
// as pairs of floats.  So the order, and with it the last bits, depend on the
// tensors' sizes, types and places within 16 bytes, and on nothing else.
//
// Sets of at most kClipClusterPieces pieces in at most 64 tensors run as one
// cluster of 8 CTAs in one launch: sums, norm and scaling.  Larger ones take a
// launch for the sums and one for the scaling, whose CTAs each form the norm
// from all CTAs' sums; the second takes the pieces in descending order, from
// those that the first left in L2.
//
// What bounds it: three passes over HBM (in, in again, out) for sets larger
// than L2.  grad_W [151936, 4096] in fp32: 7.47 GB in 1.12 ms, 6.66 TB/s, the
// rate of a plain copy; 290 ragged bf16 and fp32 tensors: 1.42 GB in 229 us,
// 6.2 TB/s; 12 tensors of 40001 elements in all: 6.6 us, latency.  Measured
// and dropped for the two large sets: one element a load 1607 and 660 us; a
// barrier after every 16384 elements 1107 and 233; warps alone on 2048
// elements 1143 and 235; one unbroken run of elements a CTA 1121 and 283.
#include <cmath>
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = kClipPieceBytes / 16 / kThreads;  // of a thread, in a piece
constexpr int kClipCluster = 8;
static_assert(kVecs == 4, "a thread's sums: two sets of four fp32, or one of eight 16-bit elements");

// A piece: bytes [lo, hi) of the 16 KB at `in`, which is 16-byte aligned and may start before the
// tensor.  `out` is the output's counterpart of `in`, 16-byte aligned too or not.
struct Piece {
    const char* in;
    char* out;
    int lo, hi, type;
};

// Piece c; `near`, the tensor that held the CTA's last piece, is tried first.
template <typename Table>
__device__ __forceinline__ Piece piece_of(const Table& t, int c, int& near) {
    if (c < t.first[near] || c >= t.first[near + 1]) {
        int lo = 0, hi = t.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (t.first[mid] <= c) lo = mid; else hi = mid - 1;
        }
        near = lo;
    }
    const ClipEntry& e = t.e[near];
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(e.in) & 15);
    const int64_t at = static_cast<int64_t>(c - t.first[near]) * kClipPieceBytes;
    const int64_t end = lead + e.n * (t.dtype[near] == RLK_DTYPE_F32 ? 4 : 2) - at;
    Piece p;
    p.in = static_cast<const char*>(e.in) - lead + at;
    p.out = static_cast<char*>(e.out) - lead + at;
    p.lo = at == 0 ? lead : 0;
    p.hi = end < kClipPieceBytes ? static_cast<int>(end) : kClipPieceBytes;
    p.type = t.dtype[near];
    return p;
}

__device__ __forceinline__ int vec_at(int m) { return (m * kThreads + static_cast<int>(threadIdx.x)) * 16; }

struct Vecs {
    uint4 v[kVecs];
    // bytes outside [lo, hi) are zero
    __device__ __forceinline__ void load(const Piece& p) {
#pragma unroll
        for (int m = 0; m < kVecs; ++m) {
            const int b = vec_at(m);
            if (b >= p.lo && b + 16 <= p.hi) {
                v[m] = *reinterpret_cast<const uint4*>(p.in + b);
            } else {
                v[m] = b < p.hi ? edge(p.in + b, p.lo - b, p.hi - b) : make_uint4(0u, 0u, 0u, 0u);
            }
        }
    }
    // the vector at q that the tensor starts or ends in: its bytes [lo, hi), kept apart from the
    // whole ones' path (arguments and result in registers)
    static __device__ __noinline__ uint4 edge(const char* q, int lo, int hi) {
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            w[r] = 4 * r >= lo && 4 * r < hi ? *reinterpret_cast<const uint16_t*>(q + 4 * r) : 0u;
            if (4 * r + 2 >= lo && 4 * r + 2 < hi)
                w[r] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(q + 4 * r + 2)) << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The two elements of a word.
template <int kType>
__device__ __forceinline__ float2 halves(uint32_t w) {
    if constexpr (kType == RLK_DTYPE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

struct Sums {
    float low[8] = {}, high[8] = {};
    template <int kType>
    __device__ __forceinline__ void add_as(const Vecs& x) {
#pragma unroll
        for (int m = 0; m < kVecs; ++m) {
            const uint32_t w[4] = {x.v[m].x, x.v[m].y, x.v[m].z, x.v[m].w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (kType == RLK_DTYPE_F32) {
                    const float f = __uint_as_float(w[r]);
                    low[(m & 1) * 4 + r] = __fmaf_rn(f, f, low[(m & 1) * 4 + r]);
                } else {
                    const float2 f = halves<kType>(w[r]);
                    low[2 * r] = __fmaf_rn(f.x, f.x, low[2 * r]);
                    low[2 * r + 1] = __fmaf_rn(f.y, f.y, low[2 * r + 1]);
                }
            }
        }
    }
    __device__ __forceinline__ void add(const Vecs& x, int type) {
        if (type == RLK_DTYPE_F32) add_as<RLK_DTYPE_F32>(x);
        else if (type == RLK_DTYPE_BF16) add_as<RLK_DTYPE_BF16>(x);
        else add_as<RLK_DTYPE_F16>(x);
    }
    __device__ __forceinline__ void empty() {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            high[r] = __fadd_rn(high[r], low[r]);
            low[r] = 0.0f;
        }
    }
    __device__ __forceinline__ float2 total() {
        empty();
#pragma unroll
        for (int n = 4; n >= 1; n >>= 1) {
#pragma unroll
            for (int i = 0; i < n; ++i) high[i] = __fadd_rn(high[2 * i], high[2 * i + 1]);
        }
        return pair_of(warp_sum(high[0]));
    }
};

// Squares of pieces c0, c0 + step, ...: the sum of the warp's.
template <typename Table>
__device__ __forceinline__ float2 sum_pieces(const Table& t, int c0, int step) {
    Sums sums;
    const int total = t.first[t.count];
    int near = 0, done = 0;
    if (c0 < total) {
        Piece p = piece_of(t, c0, near);
        Vecs x, next;
        x.load(p);
        for (int c = c0; c < total; c += step) {
            const int type = p.type;
            if (c + step < total) {
                p = piece_of(t, c + step, near);
                next.load(p);
            }
            sums.add(x, type);
            if ((++done & 15) == 0) sums.empty();
            x = next;
        }
    }
    return sums.total();
}

template <int kType>
__device__ __forceinline__ void scale_vecs(Vecs& x, float scale) {
#pragma unroll
    for (int m = 0; m < kVecs; ++m) {
        uint32_t w[4] = {x.v[m].x, x.v[m].y, x.v[m].z, x.v[m].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (kType == RLK_DTYPE_F32) {
                w[r] = __float_as_uint(__fmul_rn(__uint_as_float(w[r]), scale));
            } else {
                const float2 f = halves<kType>(w[r]);
                const float a = __fmul_rn(f.x, scale), b = __fmul_rn(f.y, scale);
                if constexpr (kType == RLK_DTYPE_BF16) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                    w[r] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                    const __half2 h = __floats2half2_rn(a, b);
                    w[r] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
        x.v[m] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ void store_piece(const Piece& p, Vecs& x, float scale) {
    if (p.type == RLK_DTYPE_F32) scale_vecs<RLK_DTYPE_F32>(x, scale);
    else if (p.type == RLK_DTYPE_BF16) scale_vecs<RLK_DTYPE_BF16>(x, scale);
    else scale_vecs<RLK_DTYPE_F16>(x, scale);
    const bool whole = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
#pragma unroll
    for (int m = 0; m < kVecs; ++m) {
        const int b = vec_at(m);
        if (whole && b >= p.lo && b + 16 <= p.hi) {
            __stcs(reinterpret_cast<uint4*>(p.out + b), x.v[m]);
        } else if (b < p.hi) {
            // the tensor starts or ends here, or the output lies differently in its 16 bytes
            const uint32_t w[4] = {x.v[m].x, x.v[m].y, x.v[m].z, x.v[m].w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = b + 4 * r;
                if (p.type == RLK_DTYPE_F32) {
                    if (i >= p.lo && i < p.hi) *reinterpret_cast<uint32_t*>(p.out + i) = w[r];
                } else {
                    if (i >= p.lo && i < p.hi) *reinterpret_cast<uint16_t*>(p.out + i) = static_cast<uint16_t>(w[r]);
                    if (i + 2 >= p.lo && i + 2 < p.hi)
                        *reinterpret_cast<uint16_t*>(p.out + i + 2) = static_cast<uint16_t>(w[r] >> 16);
                }
            }
        }
    }
}

// Pieces c0, c0 - step, ... scaled; with a scale of 1 those in place stay as they are.
template <typename Table>
__device__ __forceinline__ void scale_pieces(const Table& t, int c0, int step, float scale) {
    int near = 0;
    if (c0 < 0) return;
    Piece p = piece_of(t, c0, near);
    Vecs x, next;
    bool skip = scale == 1.0f && p.in == p.out;
    if (!skip) x.load(p);
    for (int c = c0; c >= 0; c -= step) {
        const Piece cur = p;
        const bool cur_skip = skip;
        if (c >= step) {
            p = piece_of(t, c - step, near);
            skip = scale == 1.0f && p.in == p.out;
            if (!skip) next.load(p);
        }
        if (!cur_skip) store_piece(cur, x, scale);
        x = next;
    }
}

// The limit in fp32 (a conversion from fp64 on the device is as slow as fp64 itself): an fp32 norm
// is above max_norm where it is above the largest fp32 number that is not.
struct ClipCall : ClipOut {
    float limit, max32;
};

// The sum of what eight lanes in a row hold, on each of them.
__device__ __forceinline__ float2 sum_of_8(float2 v) {
#pragma unroll 1
    for (int o = 4; o >= 1; o >>= 1)
        v = pair_add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}

// A CTA's sum from its 8 warps', on every thread.
__device__ __forceinline__ float2 warps_sum(float2 v, float2* smem) {
    static_assert(kWarps == 8, "a lane a warp");
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    return sum_of_8(smem[threadIdx.x & 7]);
}

// (norm, scale) from the sum of all squares.
__device__ __forceinline__ float2 norm_and_scale(float2 sum, const ClipCall& o) {
    const float norm = __fsqrt_rn(__fadd_rn(sum.x, sum.y));
    return make_float2(norm, norm < CUDART_INF_F && norm > o.limit ? __fdiv_rn(o.max32, norm) : 1.0f);
}
// and from the slots, by a CTA of 256 threads, each of which gets them.
__device__ __forceinline__ float2 norm_and_scale(const float2* slots, int n, const ClipCall& o, float2* smem) {
    float2 v = pair_of(0.0f);
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) v = pair_add(v, slots[i]);
    return norm_and_scale(warps_sum(warp_sum(v), smem), o);
}

__device__ __forceinline__ void write_norm(const ClipCall& o, float2 r) {
    *o.norm = r.x;
    if (o.scale) *o.scale = r.y;
    if (!(r.x < CUDART_INF_F)) report_status(o.status, RLK_ERR_NONFINITE);
}

// ---------------------------------------------------------------- one launch
__global__ void __launch_bounds__(kThreads) k_clip_cluster(const __grid_constant__ ClipTableSmall t,
                                                           const ClipCall o) {
    __shared__ float2 slots[kClipCluster];  // every CTA's sum, in every CTA
    __shared__ float2 tmp[kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank()), total = t.first[t.count];
    const float2 sum = warps_sum(sum_pieces(t, rank, kClipCluster), tmp);
    cluster.barrier_wait();  // every CTA has started: its shared memory may be written
    if (threadIdx.x < kClipCluster) cluster.map_shared_rank(slots, threadIdx.x)[rank] = sum;
    cluster.sync();
    static_assert(kClipCluster == 8, "a lane a CTA");
    const float2 res = norm_and_scale(sum_of_8(slots[threadIdx.x & 7]), o);
    if (rank == 0 && threadIdx.x == 0) write_norm(o, res);
    if (o.scale && total > rank)
        scale_pieces(t, rank + (total - 1 - rank) / kClipCluster * kClipCluster, kClipCluster, res.y);
}

// ---------------------------------------------------------------- two launches
__global__ void __launch_bounds__(kThreads, kClipCtasPerSm) k_grad_sumsq(const __grid_constant__ ClipTable t,
                                                                         float2* slots) {
    __shared__ float2 tmp[kWarps];
    ptx::grid_dependents_launch();
    const float2 sum = warps_sum(sum_pieces(t, blockIdx.x, gridDim.x), tmp);
    if (threadIdx.x == 0) slots[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) k_grad_norm(const float2* slots, int n, const ClipCall o) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o, tmp);
    if (threadIdx.x == 0) write_norm(o, r);
}

__global__ void __launch_bounds__(kThreads, kClipCtasPerSm) k_grad_scale(const __grid_constant__ ClipTable t, const float2* slots,
                                                         int n, const ClipCall o, int write) {
    __shared__ float2 tmp[kThreads / 32];
    ptx::grid_dependency_wait();
    const float2 r = norm_and_scale(slots, n, o, tmp);
    if (write && blockIdx.x == 0 && threadIdx.x == 0) write_norm(o, r);
    scale_pieces(t, t.first[t.count] - 1 - static_cast<int>(blockIdx.x), gridDim.x, r.y);
}

ClipCall call_of(const ClipOut& o) {
    ClipCall c;
    static_cast<ClipOut&>(c) = o;
    c.limit = c.max32 = static_cast<float>(o.max_norm);
    if (static_cast<double>(c.limit) > o.max_norm) c.limit = std::nextafterf(c.limit, 0.0f);
    return c;
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
    return cudaLaunchKernelEx(&cfg, k_clip_cluster, t, call_of(o));
}

cudaError_t launch_grad_sumsq(const ClipTable& t, float2* slots, cudaStream_t stream) {
    k_grad_sumsq<<<clip_launch_slots(t.first[t.count]), kThreads, 0, stream>>>(t, slots);
    return cudaGetLastError();
}

cudaError_t launch_grad_norm(const float2* slots, int n, const ClipOut& o, cudaStream_t stream) {
    return launch_after(k_grad_norm, 1, stream, slots, n, call_of(o));
}

cudaError_t launch_grad_scale(const ClipTable& t, const float2* slots, int n, const ClipOut& o, bool write,
                              cudaStream_t stream) {
    return launch_after(k_grad_scale, clip_launch_slots(t.first[t.count]), stream, t, slots, n, call_of(o), int(write));
}

}  // namespace rlk
