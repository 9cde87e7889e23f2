// Clipped policy loss with a KL term, and its gradient with respect to the
// new log-probabilities, for packed sequences.
//
// Per active token, with d = logprob - old, r = e^d, A its advantage:
//   s = min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
//   s = max(s, dual A)                     where dual > 0 and A < 0
//   k = d' | d'^2 / 2 | e^-d' - 1 + d'     with d' = logprob - ref (k1, k2, k3)
//   loss = scale sum_t w_t (-s_t + kl_coef k_t)
//   grad_t = scale w_t (-[s follows r] r A + kl_coef dk/dlogprob)
// w_t is 1, 1 / (active tokens), or 1 / (n_seqs * active tokens of t's sequence).
//
// Whether a token is clipped is decided on d itself, held exactly as two
// floats, against log(1 + clip_high) and the others as two floats: the same
// decision as in exact arithmetic (to 2^-48), where a comparison of the
// rounded ratio could go either way next to the border.
//
// The weights need counts of active tokens before the first gradient, so
// there are two passes over the mask and one over everything else.  Up to
// kClusterTokens tokens one cluster of 8 CTAs does it all in one launch, the
// counts and partial sums meeting in its shared memory; beyond, a counting
// launch is followed by one CTA per unit of 1024 tokens, the last of which
// adds up the units.  Both add the same numbers in the same order.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;               // threads of a unit
constexpr int kPer = kPolicyUnit / kThreads;
constexpr int kCluster = 8;                 // CTAs of the one-launch path
constexpr int kGroups = 4;                  // units that one of them works on at a time
constexpr int64_t kClusterTokens = 65536;   // largest batch of the one-launch path
constexpr int kClusterSeqs = 8192;          // and its most sequences (their counts in shared memory)

struct Bounds {
    int first, last;   // tokens outside [first, last) belong to no sequence
};

__device__ __forceinline__ Bounds bounds_of(const PolicyArgs& a) {
    Bounds b;
    b.first = a.offsets ? a.offsets[0] : 0;
    b.last = a.offsets ? a.offsets[a.n_seqs] : a.T;
    return b;
}

// [b, e) cut to the batch
__device__ __forceinline__ int count_active(const uint8_t* active, int64_t b, int64_t e, int T,
                                            int thread, int threads) {
    b = b < 0 ? 0 : b;
    e = e > T ? T : e;
    int n = 0;
    // bytes up to the first 16-byte boundary, 16 at a time, and the rest
    const int64_t lead = (16 - ((reinterpret_cast<uintptr_t>(active) + b) & 15)) & 15;
    const int64_t body = b + lead < e ? b + lead : e;
    const int64_t words = (e - body) / 16;
    for (int64_t t = b + thread; t < body; t += threads) n += active[t] != 0;
    for (int64_t i = thread; i < words; i += threads) {
        const uint4 v = reinterpret_cast<const uint4*>(active + body)[i];
        n += (__popc(__vcmpne4(v.x, 0u)) + __popc(__vcmpne4(v.y, 0u)) +
              __popc(__vcmpne4(v.z, 0u)) + __popc(__vcmpne4(v.w, 0u))) >> 3;
    }
    for (int64_t t = body + words * 16 + thread; t < e; t += threads) n += active[t] != 0;
    return n;
}

struct TokenTerms {
    float policy, kl, clipped, neg_d, slope;
};

__device__ __forceinline__ TokenTerms token_terms(const PolicyArgs& a, float lp, float old,
                                                  float ref, float A) {
    TokenTerms o;
    const float2 d = two_diff(lp, old);
    float r = exp_any(d.x);
    if (r < 3.0e38f) r = __fmaf_rn(r, d.y, r);
    float held = r;
    bool shut = false;
    if (A > 0.0f) {
        if (above(d, a.log_high)) {
            shut = true;
            held = a.ratio_high;
        }
    } else if (A < 0.0f) {
        if (below(d, a.log_low)) {
            shut = true;
            held = a.ratio_low;
        }
        if (a.dual > 0.0f && above(d, a.log_dual)) {
            shut = true;
            held = a.dual;
        }
    }
    float s = __fmul_rn(held, A);
    if (A == 0.0f && r == CUDART_INF_F) s = 0.0f;  // the ratio is finite, its fp32 value is not
    o.policy = -s;
    o.clipped = shut ? 1.0f : 0.0f;
    o.neg_d = -d.x;
    o.slope = shut ? 0.0f : -s;
    o.kl = 0.0f;
    if (a.ref_logprob) {
        const float u = __fsub_rn(ref, lp);
        float dk;
        if (a.kl_kind == RLK_KL_K1) {
            o.kl = -u;
            dk = 1.0f;
        } else if (a.kl_kind == RLK_KL_K2) {
            o.kl = __fmul_rn(__fmul_rn(0.5f, u), u);
            dk = -u;
        } else {
            o.kl = exp_minus_1_minus(u);
            dk = -__fadd_rn(o.kl, u);
        }
        o.slope = __fmaf_rn(a.kl_coef, dk, o.slope);
    }
    return o;
}

// One unit's tokens by one of its 8 warps: gradients out, the warp's sums of the four stats
// returned to every lane.  A warp takes 128 consecutive tokens; everything is loaded before
// anything is used, inactive tokens too (their values are dropped, never multiplied).
template <typename CountOf>
__device__ __forceinline__ float4 policy_warp(const PolicyArgs& a, int64_t unit, int warp,
                                              const Bounds& bd, float w_all, CountOf count_of) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = unit * kPolicyUnit + warp * (kPer * 32);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (t0 >= a.T) return sum;
    float lp[kPer], old[kPer], ref[kPer], adv[kPer];
    bool on[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + i * 32 + lane;
        const bool in = t < a.T;
        lp[i] = in ? a.logprob[t] : 0.0f;
        old[i] = in ? a.old_logprob[t] : 0.0f;
        ref[i] = in && a.ref_logprob ? a.ref_logprob[t] : 0.0f;
        adv[i] = in && !a.adv_per_seq ? a.advantages[t] : 0.0f;
        on[i] = in && t >= bd.first && t < bd.last && (!a.active || a.active[t] != 0);
    }
    const bool by_seq = a.offsets && (a.adv_per_seq || a.reduction == RLK_REDUCE_SEQ_MEAN);
    int seq_lo = 0, seq_hi = 0;
    if (by_seq) {
        const int64_t tl = t0 + kPer * 32 - 1;
        seq_lo = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(t0));
        seq_hi = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(tl < a.T ? tl : a.T - 1));
        if (seq_hi < seq_lo) seq_hi = seq_lo;
    }
    const float scale = static_cast<float>(a.scale);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + i * 32 + lane;
        float g = 0.0f;
        if (on[i]) {
            const int s = by_seq ? find_seq(a.offsets, seq_lo, seq_hi, static_cast<int>(t)) : 0;
            float w = w_all;
            if (a.reduction == RLK_REDUCE_SEQ_MEAN) {
                const int n = count_of(s);
                w = __fdiv_rn(1.0f, __fmul_rn(static_cast<float>(a.n_seqs),
                                              static_cast<float>(n > 1 ? n : 1)));
            }
            if (a.adv_per_seq) adv[i] = a.advantages[s];
            const TokenTerms o = token_terms(a, lp[i], old[i], ref[i], adv[i]);
            sum.x = __fmaf_rn(w, o.policy, sum.x);
            sum.y = __fmaf_rn(w, o.kl, sum.y);
            sum.z = __fmaf_rn(w, o.clipped, sum.z);
            sum.w = __fmaf_rn(w, o.neg_d, sum.w);
            g = __fmul_rn(__fmul_rn(scale, w), o.slope);
        }
        if (a.grad && t < a.T) a.grad[t] = g;
    }
    sum.x = warp_sum(sum.x);
    sum.y = warp_sum(sum.y);
    sum.z = warp_sum(sum.z);
    sum.w = warp_sum(sum.w);
    return sum;
}

// Component k of a unit's sum from its 8 warps' sums.
__device__ __forceinline__ float unit_sum(const float4* warps, int k) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v = __fadd_rn(v, reinterpret_cast<const float*>(warps + i)[k]);
    return v;
}

__device__ __forceinline__ float token_weight(const PolicyArgs& a, int n) {
    return a.reduction == RLK_REDUCE_TOKEN_MEAN ? __fdiv_rn(1.0f, static_cast<float>(n > 1 ? n : 1)) : 1.0f;
}

// Offsets that descend or leave [0, T], seen by any of `threads` threads.
__device__ __forceinline__ bool offsets_bad(const PolicyArgs& a, int thread, int threads) {
    bool bad = false;
    if (a.offsets) {
        for (int64_t s = thread; s <= a.n_seqs; s += threads) {
            const int b = a.offsets[s], e = s < a.n_seqs ? a.offsets[s + 1] : a.T;
            bad |= b < 0 || e < b || e > a.T;
        }
    }
    return bad;
}

// The loss from the units' sums, by the first 256 threads of a CTA (all of it calls).
__device__ __forceinline__ void policy_finish(const PolicyArgs& a, const float4* parts, int64_t units,
                                              bool bad, double (*smem)[4]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < kThreads) {
        double v[4] = {0.0, 0.0, 0.0, 0.0};
        for (int64_t u = threadIdx.x; u < units; u += kThreads) {
            const float4 p = parts[u];
            v[0] += static_cast<double>(p.x);
            v[1] += static_cast<double>(p.y);
            v[2] += static_cast<double>(p.z);
            v[3] += static_cast<double>(p.w);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = warp_sum(v[k]);
            if (lane == 0) smem[warp][k] = v[k];
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double s[4];
        for (int k = 0; k < 4; ++k) {
            s[k] = smem[0][k];
            for (int i = 1; i < kThreads / 32; ++i) s[k] += smem[i][k];
        }
        const float nan = CUDART_NAN_F;
        *a.out_loss = bad ? nan : static_cast<float>(a.scale * (s[0] + a.kl_coef64 * s[1]));
        for (int k = 0; k < 4; ++k) a.out_stats[k] = bad ? nan : static_cast<float>(s[k]);
        if (bad) report_status(a.status, RLK_ERR_INVALID_ARG);
    }
}

// ---------------------------------------------------------------- one launch
// Dynamic shared memory: int counts[n_seqs] (seq_mean with a mask).
__global__ void __launch_bounds__(kGroups * kThreads) k_policy_cluster(const PolicyArgs a) {
    extern __shared__ int counts[];
    __shared__ float4 parts[kClusterTokens / kPolicyUnit];   // the first CTA's are used
    __shared__ float4 warps[kGroups][kThreads / 32];
    __shared__ double finish[kThreads / 32][4];
    __shared__ int active_here;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank());
    const int lane = threadIdx.x & 31, group = threadIdx.x / kThreads;
    const int warp = (threadIdx.x % kThreads) >> 5;
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    const Bounds bd = bounds_of(a);
    const bool masked = a.active != nullptr;
    const bool by_seq = a.reduction == RLK_REDUCE_SEQ_MEAN;
    int n_all = bd.last - bd.first;
    if (masked && a.reduction != RLK_REDUCE_SUM) {
        // each CTA counts an eighth of the tokens (token_mean) or of the sequences (seq_mean)
        if (threadIdx.x == 0) active_here = 0;
        __syncthreads();
        if (by_seq) {
            cluster.barrier_wait();  // every CTA has started: its shared memory may be written
            for (int s = rank * (kGroups * kThreads / 32) + (threadIdx.x >> 5); s < a.n_seqs;
                 s += kCluster * (kGroups * kThreads / 32)) {
                const int64_t b = a.offsets ? a.offsets[s] : 0, e = a.offsets ? a.offsets[s + 1] : a.T;
                const int n = __reduce_add_sync(0xffffffffu, count_active(a.active, b, e, a.T, lane, 32));
                // every CTA keeps all counts
                if (lane < kCluster) *cluster.map_shared_rank(counts + s, lane) = n;
            }
        } else {
            int n = count_active(a.active, bd.first, bd.last, a.T,
                                 rank * (kGroups * kThreads) + threadIdx.x, kCluster * kGroups * kThreads);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0) atomicAdd(&active_here, n);
            cluster.barrier_wait();
        }
        cluster.sync();
        if (!by_seq) {
            n_all = 0;
            for (int c = 0; c < kCluster; ++c) n_all += *cluster.map_shared_rank(&active_here, c);
        }
    } else {
        cluster.barrier_wait();
    }
    const float w_all = token_weight(a, n_all);
    auto count_of = [&](int s) {
        return masked ? counts[s] : (a.offsets ? a.offsets[s + 1] - a.offsets[s] : a.T);
    };
    float4* const all_parts = cluster.map_shared_rank(parts, 0);
    for (int64_t u0 = rank * kGroups; u0 < units; u0 += kCluster * kGroups) {
        const int64_t u = u0 + group;
        const float4 s = policy_warp(a, u, warp, bd, w_all, count_of);
        if (lane == 0) warps[group][warp] = s;
        __syncthreads();
        if (threadIdx.x % kThreads < 4 && u < units)
            reinterpret_cast<float*>(all_parts + u)[threadIdx.x % kThreads] =
                unit_sum(warps[group], threadIdx.x % kThreads);
        __syncthreads();
    }
    cluster.sync();
    if (rank != 0) return;
    const bool bad = __syncthreads_or(offsets_bad(a, threadIdx.x, kGroups * kThreads));
    policy_finish(a, parts, units, bad, finish);
}

// ---------------------------------------------------------------- two launches
// Active tokens of each sequence (seq_mean) or of each block's share of all sequences
// (token_mean); and the main kernel's ticket set to 0.
__global__ void __launch_bounds__(kThreads) k_policy_count(const PolicyArgs a) {
    __shared__ int smem[kThreads / 32];
    ptx::grid_dependents_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    if (!a.active || a.reduction == RLK_REDUCE_SUM) return;
    const bool per_seq = a.reduction == RLK_REDUCE_SEQ_MEAN;
    const int rows = per_seq ? a.n_seqs : kPolicyCountBlocks;
    for (int s = blockIdx.x; s < rows; s += gridDim.x) {
        int n;
        if (per_seq) {
            n = count_active(a.active, a.offsets ? a.offsets[s] : 0, a.offsets ? a.offsets[s + 1] : a.T,
                             a.T, threadIdx.x, kThreads);
        } else {
            const Bounds bd = bounds_of(a);
            const int64_t len = static_cast<int64_t>(bd.last) - bd.first;
            const int64_t share = ((len + kPolicyCountBlocks - 1) / kPolicyCountBlocks + 15) / 16 * 16;
            const int64_t b = bd.first + s * share, e = b + share;
            n = count_active(a.active, b, e < bd.last ? e : bd.last, a.T, threadIdx.x, kThreads);
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = n;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kThreads / 32; ++i) n += smem[i];
            a.counts[s] = n;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) k_policy_main(const PolicyArgs a) {
    __shared__ float4 warps[kThreads / 32];
    __shared__ double finish[kThreads / 32][4];
    __shared__ int total;
    __shared__ bool last_here;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Bounds bd = bounds_of(a);
    if (threadIdx.x == 0) total = 0;
    ptx::grid_dependency_wait();
    __syncthreads();
    int n_all = bd.last - bd.first;
    if (a.active && a.reduction == RLK_REDUCE_TOKEN_MEAN) {
        const int n = __reduce_add_sync(0xffffffffu, a.counts[threadIdx.x]);
        if (lane == 0) atomicAdd(&total, n);
        __syncthreads();
        n_all = total;
    }
    const float w_all = token_weight(a, n_all);
    auto count_of = [&](int s) {
        return a.active ? a.counts[s] : (a.offsets ? a.offsets[s + 1] - a.offsets[s] : a.T);
    };
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const float4 s = policy_warp(a, u, warp, bd, w_all, count_of);
        if (lane == 0) warps[warp] = s;
        __syncthreads();
        if (threadIdx.x < 4) reinterpret_cast<float*>(a.parts + u)[threadIdx.x] = unit_sum(warps, threadIdx.x);
        __syncthreads();
    }
    // the last CTA to come here adds up the units
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last_here = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!last_here) return;
    __threadfence();
    const bool bad = __syncthreads_or(offsets_bad(a, threadIdx.x, kThreads));
    policy_finish(a, a.parts, units, bad, finish);
}

}  // namespace

bool policy_one_launch(int64_t T, int64_t n_seqs) {
    return T <= kClusterTokens && n_seqs <= kClusterSeqs;
}

cudaError_t launch_policy_loss(const PolicyArgs& a, int num_sms, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (policy_one_launch(a.T, a.n_seqs)) {
        cfg.gridDim = dim3(kCluster, 1, 1);
        cfg.blockDim = dim3(kGroups * kThreads, 1, 1);
        if (a.active && a.reduction == RLK_REDUCE_SEQ_MEAN) cfg.dynamicSmemBytes = size_t(a.n_seqs) * sizeof(int);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, k_policy_cluster, a);
    }
    int rows = 1;
    if (a.active && a.reduction != RLK_REDUCE_SUM)
        rows = a.reduction == RLK_REDUCE_SEQ_MEAN ? a.n_seqs : kPolicyCountBlocks;
    const int most = num_sms * 8;
    if (rows > most) rows = most;
    k_policy_count<<<rows > 0 ? rows : 1, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    cfg.gridDim = dim3(static_cast<unsigned>(units < most ? units : most), 1, 1);
    if (units == 0) cfg.gridDim.x = 1;
    cfg.blockDim = dim3(kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, k_policy_main, a);
}

}  // namespace rlk
