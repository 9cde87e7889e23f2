// Verification of drafted tokens against the target's probabilities.
//
// The rows' (m, s) pairs and lse come from the materialised-logits pass and the
// tile tree.  One cluster per sequence then decides and draws:
//
//   accept x_i while u_i q_i(x_i) < p_i(x_i), a thread per drafted token;
//   the next token is argmax_v w(v) / e(v) over row i of the first refusal, with
//   w = max(p - q, 0), or behind the last draft, with w = p.
//
// A draw by a race of exponentials is a maximum, so its result does not depend
// on how the vocabulary is split over threads and CTAs; the lowest token wins a
// tie.  p = e^(l - m) / s and q = e^(d - draft_lse) are formed from exact
// differences (a rounded value and its error), since l - m alone, rounded,
// would cost 2^-21 of p at l - m = -16.
//
// The draw reads the target's row and the noise.  A weight is at most p, so a
// token whose upper bound p / e, from the hardware's approximate exponential
// and reciprocal (2^-15 off at most above 2^-100) with 2^-10 to spare, is below
// the best weight known so far needs no closer look, and the draft's row is
// read only for those that do.
//
// What bounds it: HBM for large batches, latency for small ones.
#include <cooperative_groups.h>
#include <cstdint>

#include "rlk_block.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kAhead = 8;  // tokens that a thread loads at a time

__device__ __forceinline__ float logit_at(const void* base, int dtype, int64_t i) {
    if (dtype == RLK_DTYPE_F32) return static_cast<const float*>(base)[i];
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
}

// e^(a - b), the difference exact
__device__ __forceinline__ float exp_diff(float a, float b) {
    const float2 d = two_diff(a, b);
    const float e = exp_any(d.x);
    return __fmaf_rn(e, d.y, e);
}
__device__ __forceinline__ float approx_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float approx_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A positive weight and its token as one number: the larger weight first, then the lower token.
// 0 is no token.
__device__ __forceinline__ uint64_t key_of(float w, int token) {
    return (static_cast<uint64_t>(__float_as_uint(w)) << 32) | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ uint64_t max_key(uint64_t a, uint64_t b) { return a > b ? a : b; }

// What is drawn from: a target row, a draft row or a certain token to take off, the noise.
struct Row {
    const void* target;
    const void* draft;    // or nullptr
    const float* noise;
    int64_t target_at, draft_at, noise_at;  // the rows' first elements
    float m, s, draft_lse;
    int certain;          // token with q = 1, or -1
};

// The weight of a token, exactly as defined.
__device__ __forceinline__ float weight_of(const VerifyArgs& a, const Row& r, int v, float l, float e) {
    float w = __fdiv_rn(exp_diff(l, r.m), r.s);
    if (r.draft) w = __fsub_rn(w, exp_diff(logit_at(r.draft, a.draft_dtype, r.draft_at + v), r.draft_lse));
    else if (v == r.certain) w = __fsub_rn(w, 1.0f);
    return w > 0.0f ? __fdiv_rn(w, e) : 0.0f;
}

// The best key of tokens [v0, v1) over the CTA's threads; `best_w` (shared) is a weight that some
// token has.
__device__ uint64_t draw_range(const VerifyArgs& a, const Row& r, int v0, int v1, volatile float* best_w) {
    uint64_t best = 0;
    const float log2e = 0x1.715476p+0f;
    const float inv_s = __fmul_rn(__fdiv_rn(1.0f, r.s), 1.0f + 0x1p-10f);
    for (int base = v0; base < v1; base += kThreads * kAhead) {
        float l[kAhead], e[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int v = base + k * kThreads + static_cast<int>(threadIdx.x);
            l[k] = v < v1 ? logit_at(r.target, a.target_dtype, r.target_at + v) : -CUDART_INF_F;
            e[k] = v < v1 ? r.noise[r.noise_at + v] : 1.0f;
        }
        const float known = *best_w;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int v = base + k * kThreads + static_cast<int>(threadIdx.x);
            const float bound = __fmul_rn(__fmul_rn(approx_exp2(__fmul_rn(__fsub_rn(l[k], r.m), log2e)), inv_s),
                                          approx_rcp(e[k]));
            // a bound that is not a number, or so small that a factor may have been flushed to 0, decides
            // nothing
            if (l[k] != -CUDART_INF_F && !(bound < known && bound >= 0x1p-100f)) {
                const float w = weight_of(a, r, v, l[k], e[k]);
                if (w > 0.0f) {
                    best = max_key(best, key_of(w, v));
                    if (w > *best_w) *best_w = w;  // whichever lands is a weight that was seen
                }
            }
        }
    }
    return best;
}

__global__ void __launch_bounds__(kThreads) k_draft_verify(const VerifyArgs a) {
    __shared__ uint64_t warp_best[kThreads / 32];
    __shared__ uint64_t cta_best;
    __shared__ int first_refused;
    __shared__ float best_w;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int s = static_cast<int>(blockIdx.x) / ctas;
    ptx::grid_dependency_wait();  // the rows' pairs are the previous kernel's output
    const int o0 = a.offsets[s], o1 = a.offsets[s + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.n_draft) {
        if (rank == 0 && threadIdx.x == 0) {
            a.out_accepted[s] = -1;
            report_status(a.status, RLK_ERR_INVALID_ARG);
        }
        return;
    }
    const int n = o1 - o0;
    const int64_t row0 = static_cast<int64_t>(o0) + s;
    if (a.active && a.active[s] == 0) {
        if (rank != 0) return;
        if (threadIdx.x == 0) a.out_accepted[s] = 0;
        for (int i = threadIdx.x; i <= n; i += kThreads) {
            a.out_tokens[row0 + i] = -1;
            a.out_logprob[row0 + i] = 0.0f;
        }
        return;
    }
    if (threadIdx.x == 0) first_refused = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int x = a.tokens[o0 + i];
        bool ok = x >= 0 && x < a.V;
        if (ok) {
            const rlk_partial_t row = a.rows[row0 + i];
            const float p = __fdiv_rn(exp_diff(logit_at(a.target, a.target_dtype, (row0 + i) * a.ld_target + x), row.m), row.s);
            float q = 1.0f;
            if (a.draft)
                q = exp_diff(logit_at(a.draft, a.draft_dtype, (static_cast<int64_t>(o0) + i) * a.ld_draft + x),
                             a.draft_lse ? a.draft_lse[o0 + i] : 0.0f);
            ok = __fmul_rn(a.uniforms[o0 + i], q) < p;
        }
        if (!ok) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int acc = first_refused;
    const rlk_partial_t pair = a.rows[row0 + acc];
    Row r;
    r.target = a.target;
    r.noise = a.noise;
    r.target_at = (row0 + acc) * a.ld_target;
    r.noise_at = s * a.ld_noise;
    r.m = pair.m;
    r.s = pair.s;
    r.draft = acc < n ? a.draft : nullptr;
    r.draft_at = (static_cast<int64_t>(o0) + acc) * a.ld_draft;
    r.draft_lse = r.draft && a.draft_lse ? a.draft_lse[o0 + acc] : 0.0f;
    r.certain = acc < n && !a.draft ? a.tokens[o0 + acc] : -1;
    const int per = ((a.V + ctas - 1) / ctas + 7) / 8 * 8;
    const int v0 = min(a.V, rank * per), v1 = min(a.V, v0 + per);
    uint64_t best = 0;
    // a second time from p alone where p exceeds q nowhere
    for (int pass = 0; pass < 2 && best == 0; ++pass) {
        if (pass == 1) {
            if (acc == n) break;
            r.draft = nullptr;
            r.certain = -1;
            cluster.sync();  // everyone has read the first pass's keys
        }
        if (threadIdx.x == 0) best_w = 0.0f;
        __syncthreads();
        uint64_t mine = draw_range(a, r, v0, v1, &best_w);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mine = max_key(mine, __shfl_xor_sync(0xffffffffu, mine, o));
        if ((threadIdx.x & 31) == 0) warp_best[threadIdx.x >> 5] = mine;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kThreads / 32; ++w) mine = max_key(mine, warp_best[w]);
            cta_best = mine;
        }
        cluster.sync();
        for (int c = 0; c < ctas; ++c) best = max_key(best, *cluster.map_shared_rank(&cta_best, c));
    }
    if (rank == 0) {
        const int drawn = best != 0 ? static_cast<int>(~static_cast<uint32_t>(best)) : -1;
        for (int i = threadIdx.x; i <= n; i += kThreads) {
            const int token = i < acc ? a.tokens[o0 + i] : i == acc ? drawn : -1;
            a.out_tokens[row0 + i] = token;
            float lp = 0.0f;
            if (token >= 0)
                lp = __fsub_rn(logit_at(a.target, a.target_dtype, (row0 + i) * a.ld_target + token), a.lse[row0 + i]);
            else if (i == acc)
                lp = CUDART_NAN_F;
            a.out_logprob[row0 + i] = lp;
        }
        if (threadIdx.x == 0) {
            a.out_accepted[s] = acc;
            if (drawn < 0) report_status(a.status, RLK_ERR_NONFINITE);
            if (acc < n && (a.tokens[o0 + acc] < 0 || a.tokens[o0 + acc] >= a.V))
                report_status(a.status, RLK_ERR_TARGET_RANGE);
        }
    }
    cluster.sync();  // nobody leaves while its shared memory may be read
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& a, int num_sms, cudaStream_t stream) {
    int ctas = 8;
    while (ctas > 1 && static_cast<int64_t>(a.n_seqs) * ctas > 2 * static_cast<int64_t>(num_sms)) ctas /= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_seqs) * ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_draft_verify, a);
}

}  // namespace rlk
