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
#include "rlk_train.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = kPolicyUnit / kThreads;

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) {
    return v < lo ? lo : (v > hi ? hi : v);
}

__device__ __forceinline__ int block_sum(int v, int* smem) {
    v = __reduce_add_sync(0xffffffffu, v);
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
    for (int i = 0; i < kThreads / 32; ++i) s += smem[i];
    __syncthreads();
    return s;
}

// Active tokens of each sequence (seq_mean) or of each block's share of all
// sequences (token_mean).
__global__ void __launch_bounds__(kThreads) k_policy_count(const PolicyArgs a) {
    __shared__ int smem[kThreads / 32];
    const bool per_seq = a.reduction == RLK_REDUCE_SEQ_MEAN;
    const int rows = per_seq ? a.n_seqs : kPolicyCountBlocks;
    for (int s = blockIdx.x; s < rows; s += gridDim.x) {
        int64_t b = 0, e = a.T;
        if (per_seq) {
            if (a.offsets) {
                b = a.offsets[s];
                e = a.offsets[s + 1];
            }
        } else {
            if (a.offsets) {
                b = a.offsets[0];
                e = a.offsets[a.n_seqs];
            }
            const int64_t share = (e - b + kPolicyCountBlocks - 1) / kPolicyCountBlocks;
            const int64_t end = e;
            b += s * share;
            e = b + share < end ? b + share : end;
        }
        b = b < 0 ? 0 : b;
        e = e > a.T ? a.T : e;
        int n = 0;
        for (int64_t t = b + threadIdx.x; t < e; t += kThreads) n += a.active[t] != 0;
        n = block_sum(n, smem);
        if (threadIdx.x == 0) a.counts[s] = n;
    }
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

__global__ void __launch_bounds__(kThreads) k_policy_main(const PolicyArgs a) {
    __shared__ float smem[kThreads / 32][4];
    __shared__ int ismem[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = a.offsets ? a.offsets[0] : 0;
    const int last = a.offsets ? a.offsets[a.n_seqs] : a.T;
    float w_all = 1.0f;
    if (a.reduction == RLK_REDUCE_TOKEN_MEAN) {
        int n = a.active ? a.counts[threadIdx.x] : 0;
        n = block_sum(n, ismem);
        if (!a.active) n = last - first;
        w_all = __fdiv_rn(1.0f, static_cast<float>(n > 1 ? n : 1));
    }
    const bool need_seq = a.offsets && (a.adv_per_seq || a.reduction == RLK_REDUCE_SEQ_MEAN);
    const float scale = static_cast<float>(a.scale);
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        // a warp takes kPer * 32 consecutive tokens
        const int64_t t0 = u * kPolicyUnit + warp * (kPer * 32);
        int seq_lo = 0, seq_hi = 0;
        if (need_seq) {
            const int64_t tl = t0 + kPer * 32 - 1;
            seq_lo = warp_find_seq(a.offsets, a.n_seqs, clamp_int(static_cast<int>(t0 < a.T ? t0 : a.T - 1), 0, a.T - 1));
            seq_hi = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(tl < a.T ? tl : a.T - 1));
            if (seq_hi < seq_lo) seq_hi = seq_lo;
        }
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = t0 + i * 32 + lane;
            if (t >= a.T) continue;
            const bool on = t >= first && t < last && (!a.active || a.active[t] != 0);
            float g = 0.0f;
            if (on) {
                int s = 0;
                if (need_seq) s = find_seq(a.offsets, seq_lo, seq_hi, static_cast<int>(t));
                float w = w_all;
                if (a.reduction == RLK_REDUCE_SEQ_MEAN) {
                    const int n = a.active ? a.counts[s]
                                           : (a.offsets ? a.offsets[s + 1] - a.offsets[s] : a.T);
                    const float den = __fmul_rn(static_cast<float>(a.n_seqs), static_cast<float>(n > 1 ? n : 1));
                    w = __fdiv_rn(1.0f, den);
                }
                const float A = a.advantages[a.adv_per_seq ? s : t];
                const TokenTerms o = token_terms(a, a.logprob[t], a.old_logprob[t],
                                                 a.ref_logprob ? a.ref_logprob[t] : 0.0f, A);
                sum.x = __fmaf_rn(w, o.policy, sum.x);
                sum.y = __fmaf_rn(w, o.kl, sum.y);
                sum.z = __fmaf_rn(w, o.clipped, sum.z);
                sum.w = __fmaf_rn(w, o.neg_d, sum.w);
                g = __fmul_rn(__fmul_rn(scale, w), o.slope);
            }
            if (a.grad) a.grad[t] = g;
        }
        sum.x = warp_sum(sum.x);
        sum.y = warp_sum(sum.y);
        sum.z = warp_sum(sum.z);
        sum.w = warp_sum(sum.w);
        if (lane == 0) {
            smem[warp][0] = sum.x;
            smem[warp][1] = sum.y;
            smem[warp][2] = sum.z;
            smem[warp][3] = sum.w;
        }
        __syncthreads();
        if (threadIdx.x < 4) {
            float v = 0.0f;
            for (int i = 0; i < kThreads / 32; ++i) v = __fadd_rn(v, smem[i][threadIdx.x]);
            reinterpret_cast<float*>(a.parts + u)[threadIdx.x] = v;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) k_policy_final(const PolicyArgs a) {
    __shared__ double smem[kThreads / 32][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    if (a.offsets) {
        for (int s = threadIdx.x; s <= a.n_seqs; s += kThreads) {
            const int b = a.offsets[s], e = s < a.n_seqs ? a.offsets[s + 1] : a.T;
            bad |= b < 0 || e < b || e > a.T;
        }
    }
    bad = __syncthreads_or(bad);
    double v[4] = {0.0, 0.0, 0.0, 0.0};
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    for (int64_t u = threadIdx.x; u < units; u += kThreads) {
        const float4 p = a.parts[u];
        v[0] += static_cast<double>(p.x);
        v[1] += static_cast<double>(p.y);
        v[2] += static_cast<double>(p.z);
        v[3] += static_cast<double>(p.w);
    }
    for (int k = 0; k < 4; ++k) {
        v[k] = warp_sum(v[k]);
        if (lane == 0) smem[warp][k] = v[k];
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

}  // namespace

cudaError_t launch_policy_loss(const PolicyArgs& a, int num_sms, cudaStream_t stream) {
    if (a.T > 0 && a.n_seqs > 0 && a.active && a.reduction != RLK_REDUCE_SUM) {
        const int rows = a.reduction == RLK_REDUCE_SEQ_MEAN ? a.n_seqs : kPolicyCountBlocks;
        const int grid = rows < num_sms * 8 ? rows : num_sms * 8;
        k_policy_count<<<grid, kThreads, 0, stream>>>(a);
    }
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    const int64_t cap = static_cast<int64_t>(num_sms) * 8;
    if (units > 0)
        k_policy_main<<<static_cast<int>(units < cap ? units : cap), kThreads, 0, stream>>>(a);
    k_policy_final<<<1, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rlk
