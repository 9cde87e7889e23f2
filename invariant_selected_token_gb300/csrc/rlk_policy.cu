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
// the mask is read before anything else is formed.  Up to 4096 tokens one
// CTA, up to 32768 one cluster of 8 does it all in one launch, its threads
// holding their tokens meanwhile; beyond, a counting launch is followed by one
// CTA per unit of 1024 tokens, the last of which adds up the units.  All add
// the same numbers in the same order.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;               // threads of a unit
constexpr int kPer = kPolicyUnit / kThreads;
constexpr int kCluster = 8;                 // most CTAs of the one-launch path
constexpr int kGroups = 4;                  // units that one of them takes

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

// The tokens of one of a unit's 8 warps: 128 consecutive ones, lane l taking every 32nd.
// Everything is loaded before anything is used, inactive tokens too (their values are dropped,
// never multiplied).
struct WarpTokens {
    int64_t t0;
    float lp[kPer], old[kPer], ref[kPer], adv[kPer];
    bool on[kPer];
    __device__ __forceinline__ int64_t token(int i) const { return t0 + i * 32 + (threadIdx.x & 31); }
    __device__ __forceinline__ void load(const PolicyArgs& a, int64_t unit, int warp) {
        t0 = unit * kPolicyUnit + warp * (kPer * 32);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = token(i);
            const bool in = t < a.T;
            lp[i] = in ? a.logprob[t] : 0.0f;
            old[i] = in ? a.old_logprob[t] : 0.0f;
            ref[i] = in && a.ref_logprob ? a.ref_logprob[t] : 0.0f;
            adv[i] = in && !a.adv_per_seq ? a.advantages[t] : 0.0f;
            on[i] = in && (!a.active || a.active[t] != 0);
        }
    }
    // tokens of no sequence take no part
    __device__ __forceinline__ void cut(const Bounds& b) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) on[i] = on[i] && token(i) >= b.first && token(i) < b.last;
    }
};

// Gradients of a warp's tokens out; its sums of the four stats, on every lane.  seq_of(i) is
// token i's sequence, count_of(s) and adv_of(s) that one's active tokens and advantage.
template <typename SeqOf, typename CountOf, typename AdvOf>
__device__ __forceinline__ float4 policy_warp(const PolicyArgs& a, const WarpTokens& k, float w_all, SeqOf seq_of,
                                              CountOf count_of, AdvOf adv_of) {
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float scale = static_cast<float>(a.scale);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        float g = 0.0f;
        if (k.on[i]) {
            float w = w_all, adv = k.adv[i];
            if (a.reduction == RLK_REDUCE_SEQ_MEAN) {
                const int n = count_of(seq_of(i));
                w = __fdiv_rn(1.0f, __fmul_rn(static_cast<float>(a.n_seqs), static_cast<float>(n > 1 ? n : 1)));
            }
            if (a.adv_per_seq) adv = adv_of(seq_of(i));
            const TokenTerms o = token_terms(a, k.lp[i], k.old[i], k.ref[i], adv);
            sum.x = __fmaf_rn(w, o.policy, sum.x);
            sum.y = __fmaf_rn(w, o.kl, sum.y);
            sum.z = __fmaf_rn(w, o.clipped, sum.z);
            sum.w = __fmaf_rn(w, o.neg_d, sum.w);
            g = __fmul_rn(__fmul_rn(scale, w), o.slope);
        }
        if (a.grad && k.token(i) < a.T) a.grad[k.token(i)] = g;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        sum.x = __fadd_rn(sum.x, __shfl_xor_sync(0xffffffffu, sum.x, o));
        sum.y = __fadd_rn(sum.y, __shfl_xor_sync(0xffffffffu, sum.y, o));
        sum.z = __fadd_rn(sum.z, __shfl_xor_sync(0xffffffffu, sum.z, o));
        sum.w = __fadd_rn(sum.w, __shfl_xor_sync(0xffffffffu, sum.w, o));
    }
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

// The units' sums are added like this: slot j takes units j, j + 256, ... in ascending order, the
// 32 slots of a warp are added by a shuffle tree, the 8 warps' sums in order, all in fp64.
__device__ __forceinline__ void write_stat(const PolicyArgs& a, int k, double v, bool bad) {
    a.out_stats[k] = bad ? CUDART_NAN_F : static_cast<float>(v);
}
__device__ __forceinline__ void write_loss(const PolicyArgs& a, double policy, double kl, bool bad) {
    *a.out_loss = bad ? CUDART_NAN_F : static_cast<float>(a.scale * (policy + a.kl_coef64 * kl));
    if (bad) report_status(a.status, RLK_ERR_INVALID_ARG);
}

// ---------------------------------------------------------------- one launch
constexpr int kLaunchSeqs = 1024;  // most sequences of the one-launch path: kept in shared memory

// The last s in [0, n) with offsets[s] <= t, in shared memory.
__device__ __forceinline__ int seq_in(const int32_t* offsets, int n, int t) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One cluster of kCtas CTAs, 4 units each: a thread holds its 4 tokens from the first load to
// the gradient, and the counts that the weights need come from the masks it holds.
template <int kCtas>
__global__ void __launch_bounds__(kGroups * kThreads) k_policy_one(const PolicyArgs a) {
    constexpr int kAll = kGroups * kThreads;
    static_assert(kCtas * kGroups <= 32, "a lane per unit");
    __shared__ int32_t offsets[kLaunchSeqs + 1];
    __shared__ float adv[kLaunchSeqs];
    __shared__ int counts[kLaunchSeqs];
    __shared__ int totals[kLaunchSeqs];
    __shared__ float4 parts[32];           // the first CTA's are used
    __shared__ float4 warps[kGroups][kThreads / 32];
    __shared__ int active_here;
    const int rank = kCtas > 1 ? static_cast<int>(blockIdx.x) : 0;
    const int lane = threadIdx.x & 31, group = threadIdx.x / kThreads;
    const int warp = (threadIdx.x % kThreads) >> 5;
    const int unit = rank * kGroups + group;
    WarpTokens k;
    k.load(a, unit, warp);
    const bool masked = a.active != nullptr, by_mean = a.reduction == RLK_REDUCE_SEQ_MEAN;
    const bool by_seq = a.offsets && (a.adv_per_seq || by_mean);
    Bounds bd = {0, a.T};
    bool bad = false;
    if (a.offsets) {
        bd = bounds_of(a);
        for (int s = threadIdx.x; s <= a.n_seqs; s += kAll) {
            const int b = a.offsets[s], e = s < a.n_seqs ? a.offsets[s + 1] : a.T;
            bad |= b < 0 || e < b || e > a.T;
            offsets[s] = b;
        }
    }
    for (int s = threadIdx.x; s < a.n_seqs; s += kAll) {
        counts[s] = 0;
        if (a.adv_per_seq) adv[s] = a.advantages[s];
    }
    if (threadIdx.x == 0) active_here = 0;
    bad = __syncthreads_or(bad);
    k.cut(bd);
    int seq[kPer] = {};
    if (by_seq) {
        // a warp's 128 tokens: mostly of one sequence
        const int64_t tl = k.t0 + kPer * 32 - 1;
        const int lo = k.t0 < a.T ? seq_in(offsets, a.n_seqs, static_cast<int>(k.t0)) : 0;
        const int hi = k.t0 < a.T ? seq_in(offsets, a.n_seqs, static_cast<int>(tl < a.T ? tl : a.T - 1)) : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            seq[i] = lo;
            if (hi > lo && k.on[i]) seq[i] = lo + seq_in(offsets + lo, hi - lo + 1, static_cast<int>(k.token(i)));
        }
    }
    int n_all = bd.last - bd.first;
    if (masked && a.reduction != RLK_REDUCE_SUM) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int n = __popc(__ballot_sync(0xffffffffu, k.on[i]));
            const int s0 = __shfl_sync(0xffffffffu, seq[i], 0);
            if (!by_mean) {
                if (lane == 0 && n) atomicAdd(&active_here, n);
            } else if (__all_sync(0xffffffffu, seq[i] == s0)) {
                if (lane == 0 && n) atomicAdd(&counts[s0], n);
            } else if (k.on[i]) {
                atomicAdd(&counts[seq[i]], 1);
            }
        }
        if constexpr (kCtas > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            if (by_mean) {
                for (int s = threadIdx.x; s < a.n_seqs; s += kAll) {
                    int n = 0;
#pragma unroll
                    for (int c = 0; c < kCtas; ++c) n += cluster.map_shared_rank(counts, c)[s];
                    totals[s] = n;
                }
                __syncthreads();
            } else {
                n_all = __reduce_add_sync(0xffffffffu, lane < kCtas ? *cluster.map_shared_rank(&active_here, lane % kCtas) : 0);
            }
        } else {
            __syncthreads();
            n_all = active_here;
        }
    } else if constexpr (kCtas > 1) {
        cg::this_cluster().sync();  // every CTA has started: its shared memory may be written
    }
    const float4 s = policy_warp(
        a, k, token_weight(a, n_all), [&](int i) { return seq[i]; },
        [&](int q) {
            return masked ? (kCtas > 1 ? totals[q] : counts[q]) : (a.offsets ? offsets[q + 1] - offsets[q] : a.T);
        },
        [&](int q) { return adv[q]; });
    if (lane == 0) warps[group][warp] = s;
    __syncthreads();
    float4* all_parts = parts;
    if constexpr (kCtas > 1) all_parts = cg::this_cluster().map_shared_rank(parts, 0);
    if (threadIdx.x % kThreads < 4)
        reinterpret_cast<float*>(all_parts + unit)[threadIdx.x % kThreads] =
            unit_sum(warps[group], threadIdx.x % kThreads);
    if constexpr (kCtas > 1) cg::this_cluster().sync(); else __syncthreads();
    if (rank != 0 || threadIdx.x >= 3 * 32) return;
    // units 0 .. 31 are the first warp's slots of the order above; the rest of it adds zeros.
    // Warp 0 forms the loss and the two stats in it, warps 1 and 2 the others.
    const float* p = reinterpret_cast<const float*>(parts + lane);
    const bool have = lane < kCtas * kGroups;
    const int w = threadIdx.x >> 5;
    const double v = warp_sum(have ? static_cast<double>(p[w == 0 ? 0 : w + 1]) : 0.0);
    if (w == 0) {
        const double kl = warp_sum(have ? static_cast<double>(p[1]) : 0.0);
        if (lane == 0) {
            write_loss(a, v, kl, bad);
            write_stat(a, 0, v, bad);
            write_stat(a, 1, kl, bad);
        }
    } else if (lane == 0) {
        write_stat(a, w + 1, v, bad);
    }
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
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    WarpTokens k;
    k.load(a, blockIdx.x, warp);
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
    const bool by_seq = a.offsets && (a.adv_per_seq || a.reduction == RLK_REDUCE_SEQ_MEAN);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        if (u != blockIdx.x) k.load(a, u, warp);
        k.cut(bd);
        int seq[kPer] = {};
        if (by_seq && k.t0 < a.T) {
            const int64_t tl = k.t0 + kPer * 32 - 1;
            const int lo = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(k.t0));
            const int hi = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(tl < a.T ? tl : a.T - 1));
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                seq[i] = hi > lo && k.on[i] ? find_seq(a.offsets, lo, hi, static_cast<int>(k.token(i))) : lo;
        }
        const float4 s = policy_warp(
            a, k, w_all, [&](int i) { return seq[i]; },
            [&](int q) {
                return a.active ? a.counts[q] : (a.offsets ? a.offsets[q + 1] - a.offsets[q] : a.T);
            },
            [&](int q) { return a.advantages[q]; });
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
    bool bad = false;
    if (a.offsets) {
        for (int64_t s = threadIdx.x; s <= a.n_seqs; s += kThreads) {
            const int b = a.offsets[s], e = s < a.n_seqs ? a.offsets[s + 1] : a.T;
            bad |= b < 0 || e < b || e > a.T;
        }
    }
    bad = __syncthreads_or(bad);
    double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
        const float4 p = a.parts[u];
        v[0] += static_cast<double>(p.x);
        v[1] += static_cast<double>(p.y);
        v[2] += static_cast<double>(p.z);
        v[3] += static_cast<double>(p.w);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = __dadd_rn(v[c], __shfl_xor_sync(0xffffffffu, v[c], o));
    }
    if (lane == 0) {
        for (int c = 0; c < 4; ++c) finish[warp][c] = v[c];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        double s = finish[0][threadIdx.x];
        for (int i = 1; i < kThreads / 32; ++i) s = __dadd_rn(s, finish[i][threadIdx.x]);
        write_stat(a, threadIdx.x, s, bad);
        const double kl = __shfl_sync(0xfu, s, 1);
        if (threadIdx.x == 0) write_loss(a, s, kl, bad);
    }
}

template <int kCtas>
cudaError_t launch_one(const PolicyArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.gridDim = dim3(kCtas, 1, 1);
    cfg.blockDim = dim3(kGroups * kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCtas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_policy_one<kCtas>, a);
}

}  // namespace

bool policy_one_launch(int64_t T, int64_t n_seqs) {
    return T <= kCluster * kGroups * kPolicyUnit && n_seqs <= kLaunchSeqs;
}

cudaError_t launch_policy_loss(const PolicyArgs& a, int num_sms, cudaStream_t stream) {
    if (policy_one_launch(a.T, a.n_seqs))
        return a.T <= kGroups * kPolicyUnit ? launch_one<1>(a, stream) : launch_one<kCluster>(a, stream);
    int rows = 1;
    if (a.active && a.reduction != RLK_REDUCE_SUM)
        rows = a.reduction == RLK_REDUCE_SEQ_MEAN ? a.n_seqs : kPolicyCountBlocks;
    const int most = num_sms * 8;
    if (rows > most) rows = most;
    k_policy_count<<<rows > 0 ? rows : 1, kThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(units < most ? (units > 0 ? units : 1) : most), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_policy_main, a);
}

}  // namespace rlk
