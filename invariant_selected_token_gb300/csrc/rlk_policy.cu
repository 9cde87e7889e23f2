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
// the mask is read before anything else is formed.  Up to 1024 tokens one
// CTA, up to 32768 one cluster of 8 does it all in one launch, its threads
// holding their tokens (one up to 8192, else four) meanwhile; beyond, a
// counting launch is followed by up to four CTAs per SM, which take units of
// 1024 tokens in turn, and the last to end adds up the units.  All add the same
// numbers in the same order: a unit is 8 spans of 128 consecutive tokens; lane
// l of a span adds RN(w x) of tokens 4 l .. 4 l + 3 pairwise, the lanes a
// shuffle tree, the spans in order, all in fp32: at most 16 roundings of the
// sum of the absolute terms, next to the dozen that each term has.  The units
// are added as pairs of floats.
//
// What bounds it: latency.  4.0 us a call on the device at 512 tokens, 5.4 at
// 8192, of which one launch, one round trip to memory and the first fetch of
// the code make most.  At 1.77 M tokens (37 MB, 5.6 us of HBM) 15.4 us: 2 us of
// the counting launch that nothing hides, 3 of the last CTA's tail, and between
// them three units a CTA, each load, terms, barrier one after the other.  Its 8
// warps a scheduler use 56 % of the issue slots (cold caches); for every issue
// 3.8 warps wait for a load, 2.0 for an operation's fixed latency, 1.8 at the
// unit's barrier, 0.9 for a full pipe.  Sums in fp64
// instead of pairs of floats made it 27, the branching form of a token 23, a
// look-up of both ends of a warp's span and of every token 19.7, tokens loaded one
// by one 18.8 us.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;               // threads that a unit's sums are added by
constexpr int kUnitWarps = kThreads / 32;
constexpr int kCluster = 8;                 // most CTAs of the one-launch path
// CTAs of the main kernel per SM, all resident.  At 1.77 M tokens: 3 17.2, 4 16.1, 5 (spilling)
// 17.2 us a call.  Loading the next unit ahead, into registers or shared memory, costs 1 us.
constexpr int kMainCtasPerSm = 4;

struct PolicyCall : PolicyArgs {
    bool wide;      // four tokens' values can be loaded and stored at a time
    float2 scale2, coef2;  // scale and kl_coef, for the loss; a gradient takes their first parts,
                           // one rounding among its dozen
};

struct Bounds {
    int first, last;   // tokens outside [first, last) belong to no sequence
};

__device__ __forceinline__ Bounds bounds_of(const PolicyCall& a) {
    Bounds b;
    b.first = a.offsets ? a.offsets[0] : 0;
    b.last = a.offsets ? a.offsets[a.n_seqs] : a.T;
    return b;
}

// Active tokens of [b, e), cut to the batch, by `threads` threads.
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
#pragma unroll 4
    for (int64_t i = thread; i < words; i += threads) {
        const uint4 v = reinterpret_cast<const uint4*>(active + body)[i];
        n += (__popc(__vcmpne4(v.x, 0u)) + __popc(__vcmpne4(v.y, 0u)) +
              __popc(__vcmpne4(v.z, 0u)) + __popc(__vcmpne4(v.w, 0u))) >> 3;
    }
    for (int64_t t = body + words * 16 + thread; t < e; t += threads) n += active[t] != 0;
    return n;
}

// kKl: 0 without a reference, else RLK_KL_K1 .. K3.
struct TokenTerms {
    float policy, kl, clipped, neg_d, slope;
};

// From d as two floats, r = e^d, u = ref - lp and (k3) e^u - 1 - u.  The two clips are one test:
// with a negative advantage both d and the border change sign.  An advantage of 0 or NaN is not
// clipped.
template <int kKl>
__device__ __forceinline__ TokenTerms token_terms(const PolicyCall& a, float2 d, float r, float u, float k3, float A) {
    TokenTerms o;
    const bool up = A > 0.0f;
    const float2 side = up ? d : make_float2(-d.x, -d.y);
    const float2 border = up ? a.log_high : make_float2(-a.log_low.x, -a.log_low.y);
    bool shut = above(side, border) && fabsf(A) > 0.0f;
    float held = shut ? (up ? a.ratio_high : a.ratio_low) : r;
    if (a.dual > 0.0f && A < 0.0f && above(d, a.log_dual)) {
        shut = true;
        held = a.dual;
    }
    const float s = __fmul_rn(held, A);
    o.policy = -s;
    o.clipped = shut ? 1.0f : 0.0f;
    o.neg_d = -d.x;
    o.slope = shut ? 0.0f : -s;
    o.kl = 0.0f;
    if constexpr (kKl != 0) {
        const float dk = kKl == RLK_KL_K1 ? 1.0f : kKl == RLK_KL_K2 ? -u : -__fadd_rn(k3, u);
        o.kl = kKl == RLK_KL_K1 ? -u : kKl == RLK_KL_K2 ? __fmul_rn(__fmul_rn(0.5f, u), u) : k3;
        if (a.kl_coef != 0.0f) o.slope = __fmaf_rn(a.kl_coef, dk, o.slope);  // else k may overflow unharmed
    }
    return o;
}

// e^(d.x + d.y): the rest of d to first order.
__device__ __forceinline__ float ratio_of(float2 d) {
    const float r = exp_any(d.x);
    return r < CUDART_INF_F ? __fmaf_rn(r, d.y, r) : r;
}

// One token.
template <int kKl>
__device__ __forceinline__ TokenTerms token_one(const PolicyCall& a, float lp, float old, float ref, float A) {
    const float2 d = two_diff(lp, old);
    // u is rounded, unlike d: nothing is decided by it, and e^u is off by |u| 2^-24 of itself
    const float u = __fsub_rn(ref, lp);
    float r = ratio_of(d);
    // a ratio that is finite but beyond fp32 makes nothing of an advantage of 0
    if (A == 0.0f && r == CUDART_INF_F && fabsf(lp) < CUDART_INF_F && fabsf(old) < CUDART_INF_F) r = 1.0f;
    return token_terms<kKl>(a, d, r, u, kKl == RLK_KL_K3 ? exp_minus_1_minus(u) : 0.0f, A);
}

// Two tokens, two per instruction as far as the values allow: |d| <= 80, where 2^n only adds to
// an exponent, and |u| < 1.  The same operations in the same order, so the same bits as
// token_one; warps with other values in them run that.
template <int kKl>
__device__ __forceinline__ void token_two(const PolicyCall& a, const float (&lp)[2], const float (&old)[2],
                                          const float (&ref)[2], const float (&A)[2], TokenTerms (&o)[2]) {
    const uint64_t l2 = f2_pack(lp[0], lp[1]);
    const uint64_t neg_old = f2_pack(-old[0], -old[1]);
    const uint64_t s = f2_add(l2, neg_old);
    const uint64_t minus = f2_splat(-1.0f);
    // two_diff: t = s - lp, e = (lp - (s - t)) - (old + t); products with -1 are exact
    const uint64_t t = f2_fma(l2, minus, s);
    const uint64_t e = f2_add(f2_fma(f2_fma(t, minus, s), minus, l2), f2_fma(t, minus, neg_old));
    float d0, d1, e0, e1, u0 = 0.0f, u1 = 0.0f;
    f2_unpack(s, d0, d1);
    f2_unpack(e, e0, e1);
    bool plain = fabsf(d0) <= 80.0f && fabsf(d1) <= 80.0f;
    uint64_t u2 = 0;
    if constexpr (kKl != 0) {
        u2 = f2_fma(l2, minus, f2_pack(ref[0], ref[1]));
        f2_unpack(u2, u0, u1);
        if constexpr (kKl == RLK_KL_K3) plain = plain && fabsf(u0) < 1.0f && fabsf(u1) < 1.0f;
    }
    if (!__all_sync(0xffffffffu, plain)) {
        o[0] = token_one<kKl>(a, lp[0], old[0], ref[0], A[0]);
        o[1] = token_one<kKl>(a, lp[1], old[1], ref[1], A[1]);
        return;
    }
    uint64_t r = contract_exp_x2<false>(s);
    r = f2_fma(r, e, r);
    float r0, r1, k0 = 0.0f, k1 = 0.0f;
    f2_unpack(r, r0, r1);
    if constexpr (kKl == RLK_KL_K3) {
        uint64_t p = f2_splat(exp_tail(0));
#pragma unroll
        for (int i = 1; i < kExpTail; ++i) p = f2_fma(p, u2, f2_splat(exp_tail(i)));
        f2_unpack(f2_mul(f2_mul(u2, u2), p), k0, k1);
    }
    o[0] = token_terms<kKl>(a, make_float2(d0, e0), r0, u0, k0, A[0]);
    o[1] = token_terms<kKl>(a, make_float2(d1, e1), r1, u1, k1, A[1]);
}

// A lane's token, or four consecutive ones.  Everything is loaded before anything is used, inactive
// tokens too (their values are dropped, never multiplied).
template <int kKl, int kPer>
struct Tokens {
    int64_t t0;  // the first one
    int left;    // tokens from it to the end of the batch
    float lp[kPer], old[kPer], ref[kPer], adv[kPer];
    bool on[kPer];
    __device__ __forceinline__ bool whole(const PolicyCall& a) const { return kPer == 4 && a.wide && left >= 4; }
    __device__ __forceinline__ void load(const PolicyCall& a, int64_t first) {
        t0 = first;
        left = first < a.T ? static_cast<int>(a.T - first) : 0;
        const float *p_lp = a.logprob + t0, *p_old = a.old_logprob + t0;
        const float *p_ref = a.ref_logprob + t0, *p_adv = a.advantages + t0;
        const uint8_t* p_on = a.active + t0;
        if constexpr (kPer == 4) {
            if (whole(a)) {
                load4(lp, p_lp);
                load4(old, p_old);
                if (kKl) load4(ref, p_ref);
                if (!a.adv_per_seq) load4(adv, p_adv);
                else adv[0] = adv[1] = adv[2] = adv[3] = 0.0f;
                const uint32_t m = a.active ? *reinterpret_cast<const uint32_t*>(p_on) : 0x01010101u;
#pragma unroll
                for (int i = 0; i < 4; ++i) on[i] = (m & (0xFFu << (8 * i))) != 0;
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool in = i < left;
            lp[i] = in ? p_lp[i] : 0.0f;
            old[i] = in ? p_old[i] : 0.0f;
            ref[i] = kKl && in ? p_ref[i] : 0.0f;
            adv[i] = in && !a.adv_per_seq ? p_adv[i] : 0.0f;
            on[i] = in && (!a.active || p_on[i] != 0);
        }
    }
    static __device__ __forceinline__ void load4(float (&v)[kPer], const float* p) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    }
    // tokens of no sequence take no part
    __device__ __forceinline__ void cut(const Bounds& b) {
        if (b.first <= t0 && b.last - t0 >= kPer) return;
#pragma unroll
        for (int i = 0; i < kPer; ++i) on[i] = on[i] && t0 + i >= b.first && t0 + i < b.last;
    }
};

// Gradients of a lane's tokens out, and RN(w x) of the four stats x returned.  Every token is
// worked on, the inactive ones with zeros for their values, so that the tokens' chains of
// operations overlap; what an inactive one gives is dropped.
template <int kKl, int kPer>
__device__ __forceinline__ void policy_tokens(const PolicyCall& a, const Tokens<kKl, kPer>& k, const float (&w)[kPer],
                                              float4 (&out)[kPer]) {
    const float scale = a.scale2.x;
    float g[kPer];
    constexpr int kStep = kPer == 1 ? 1 : 2;
#pragma unroll
    for (int i = 0; i < kPer; i += kStep) {
        TokenTerms o[kStep];
        float lp[kStep], old[kStep], ref[kStep], adv[kStep];
#pragma unroll
        for (int c = 0; c < kStep; ++c) {
            const bool on = k.on[i + c];
            lp[c] = on ? k.lp[i + c] : 0.0f;
            old[c] = on ? k.old[i + c] : 0.0f;
            ref[c] = on ? k.ref[i + c] : 0.0f;
            adv[c] = on ? k.adv[i + c] : 0.0f;
        }
        if constexpr (kStep == 1) o[0] = token_one<kKl>(a, lp[0], old[0], ref[0], adv[0]);
        else token_two<kKl>(a, lp, old, ref, adv, o);
#pragma unroll
        for (int c = 0; c < kStep; ++c) {
            // an inactive token's four terms are zeros, and its weight is finite
            const float wi = w[i + c];
            float4& x = out[i + c];
            f2_unpack(f2_mul(f2_splat(wi), f2_pack(o[c].policy, o[c].kl)), x.x, x.y);
            f2_unpack(f2_mul(f2_splat(wi), f2_pack(o[c].clipped, o[c].neg_d)), x.z, x.w);
            g[i + c] = k.on[i + c] ? __fmul_rn(__fmul_rn(scale, wi), o[c].slope) : 0.0f;
        }
    }
    if (!a.grad) return;
    float* const grad = a.grad + k.t0;
    if constexpr (kPer == 4) {
        if (k.whole(a)) {
            *reinterpret_cast<float4*>(grad) = make_float4(g[0], g[1], g[2], g[3]);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (i < k.left) grad[i] = g[i];
}

struct Stats {  // (policy, kl) and (clipped, -d)
    uint64_t a, b;
};
__device__ __forceinline__ Stats stats_of(const float4& v) { return {f2_pack(v.x, v.y), f2_pack(v.z, v.w)}; }
__device__ __forceinline__ Stats add_stats(const Stats& x, const Stats& y) { return {f2_add(x.a, y.a), f2_add(x.b, y.b)}; }

// A span's sum from its lanes' four tokens.
__device__ __forceinline__ float4 span_sum(const float4& p0, const float4& p1, const float4& p2, const float4& p3) {
    Stats v = add_stats(add_stats(stats_of(p0), stats_of(p1)), add_stats(stats_of(p2), stats_of(p3)));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v = add_stats(v, {__shfl_xor_sync(0xffffffffu, v.a, o), __shfl_xor_sync(0xffffffffu, v.b, o)});
    float4 f;
    f2_unpack(v.a, f.x, f.y);
    f2_unpack(v.b, f.z, f.w);
    return f;
}

// Component k of a unit's sum from its 8 spans' sums.
__device__ __forceinline__ float unit_sum(const float4* spans, int k) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kUnitWarps; ++i) v = __fadd_rn(v, reinterpret_cast<const float*>(spans + i)[k]);
    return v;
}

// Weight of the tokens of a sequence with n active ones.
__device__ __forceinline__ float seq_weight(const PolicyCall& a, int n) {
    return __fdiv_rn(1.0f, __fmul_rn(static_cast<float>(a.n_seqs), static_cast<float>(n > 1 ? n : 1)));
}
__device__ __forceinline__ float token_weight(const PolicyCall& a, int n) {
    return a.reduction == RLK_REDUCE_TOKEN_MEAN ? __fdiv_rn(1.0f, static_cast<float>(n > 1 ? n : 1)) : 1.0f;
}

// The units' sums are added like this: slot j takes units j, j + 256, ... in ascending order, the
// 32 slots of a warp are added by a shuffle tree, the 8 warps' sums by another, all as pairs.
__device__ __forceinline__ void write_stat(const PolicyCall& a, int k, float2 v, bool bad) {
    a.out_stats[k] = bad ? CUDART_NAN_F : __fadd_rn(v.x, v.y);
}
__device__ __forceinline__ void write_loss(const PolicyCall& a, float2 policy, float2 kl, bool bad) {
    // in fp64 this would be 0.3 us of dependent operations
    const float2 sum = a.coef2.x != 0.0f ? pair_add(policy, pair_mul(a.coef2, kl)) : policy;
    *a.out_loss = bad ? CUDART_NAN_F : pair_mul(a.scale2, sum).x;
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

// One cluster of kCtas CTAs of 1024 threads, kPer tokens a thread, which it holds from the first
// load to the gradient; the counts that the weights need come from the masks it holds.
template <int kKl, int kCtas, int kPer>
__global__ void __launch_bounds__(1024) k_policy_one(const PolicyCall a) {
    constexpr int kAll = 1024, kUnits = kPer;  // units of a CTA
    static_assert(kCtas * kUnits <= 32, "a lane per unit");
    static_assert(kPer == 1 || kPer == 4, "a warp is a quarter of a span, or one");
    __shared__ int32_t offsets[kLaunchSeqs + 1];
    __shared__ float adv[kLaunchSeqs];
    __shared__ int counts[kLaunchSeqs];
    __shared__ float weights[kLaunchSeqs];
    __shared__ float4 parts[32];           // the first CTA's are used
    __shared__ float4 spans[kUnits * kUnitWarps];
    __shared__ float4 tokens[kPer == 1 ? kUnitWarps : 1][4][34];  // [span][token mod 4][lane]
    __shared__ int active_here;
    const int rank = kCtas > 1 ? static_cast<int>(blockIdx.x) : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Tokens<kKl, kPer> k;
    k.load(a, static_cast<int64_t>(rank * kAll + threadIdx.x) * kPer);
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
        // a warp's tokens: mostly of one sequence
        const int64_t tf = k.t0 - lane * kPer, tl = tf + kPer * 32 - 1;
        const int lo = tf < a.T ? seq_in(offsets, a.n_seqs, static_cast<int>(tf)) : 0;
        const int hi = tf < a.T ? seq_in(offsets, a.n_seqs, static_cast<int>(tl < a.T ? tl : a.T - 1)) : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            seq[i] = lo;
            if (hi > lo && k.on[i]) seq[i] = lo + seq_in(offsets + lo, hi - lo + 1, static_cast<int>(k.t0) + i);
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
    }
    if constexpr (kCtas > 1) {
        // the counts are complete, and every CTA has started: its shared memory may be written
        cg::this_cluster().sync();
        if (masked && a.reduction == RLK_REDUCE_TOKEN_MEAN)
            n_all = __reduce_add_sync(
                0xffffffffu, lane < kCtas ? *cg::this_cluster().map_shared_rank(&active_here, lane % kCtas) : 0);
    } else {
        __syncthreads();
        if (masked && a.reduction == RLK_REDUCE_TOKEN_MEAN) n_all = active_here;
    }
    if (by_mean) {
        for (int s = threadIdx.x; s < a.n_seqs; s += kAll) {
            int n = a.offsets ? offsets[s + 1] - offsets[s] : a.T;
            if (masked) {
                n = counts[s];
                if constexpr (kCtas > 1) {
                    n = 0;
#pragma unroll
                    for (int c = 0; c < kCtas; ++c) n += cg::this_cluster().map_shared_rank(counts, c)[s];
                }
            }
            weights[s] = seq_weight(a, n);
        }
        __syncthreads();
    }
    float w[kPer];
    const float w_all = token_weight(a, n_all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        w[i] = by_mean && a.n_seqs > 0 ? weights[seq[i]] : w_all;
        if (a.adv_per_seq) k.adv[i] = adv[seq[i]];
    }
    float4 terms[kPer];
    policy_tokens<kKl>(a, k, w, terms);
    if constexpr (kPer == 4) {
        const float4 s = span_sum(terms[0], terms[1], terms[2], terms[3]);
        if (lane == 0) spans[warp] = s;
    } else {
        tokens[threadIdx.x >> 7][threadIdx.x & 3][(threadIdx.x & 127) >> 2] = terms[0];
        __syncthreads();
        if (warp < kUnitWarps) {
            const float4(*const p)[34] = tokens[warp];
            const float4 s = span_sum(p[0][lane], p[1][lane], p[2][lane], p[3][lane]);
            if (lane == 0) spans[warp] = s;
        }
    }
    __syncthreads();
    float4* all_parts = parts;
    if constexpr (kCtas > 1) all_parts = cg::this_cluster().map_shared_rank(parts, 0);
    if (threadIdx.x < 4 * kUnits)
        reinterpret_cast<float*>(all_parts + rank * kUnits)[threadIdx.x] =
            unit_sum(spans + threadIdx.x / 4 * kUnitWarps, threadIdx.x % 4);
    if constexpr (kCtas > 1) cg::this_cluster().sync(); else __syncthreads();
    if (rank != 0 || threadIdx.x >= 3 * 32) return;
    // units 0 .. 31 are the first warp's slots of the order above; the rest of it adds zeros.
    // Warp 0 forms the loss and the two stats in it, warps 1 and 2 the others.
    const float* p = reinterpret_cast<const float*>(parts + lane);
    const bool have = lane < kCtas * kUnits;
    const int which = threadIdx.x >> 5;
    const float2 v = warp_sum(pair_of(have ? p[which == 0 ? 0 : which + 1] : 0.0f));
    if (which == 0) {
        const float2 kl = warp_sum(pair_of(have ? p[1] : 0.0f));
        if (lane == 0) {
            write_loss(a, v, kl, bad);
            write_stat(a, 0, v, bad);
            write_stat(a, 1, kl, bad);
        }
    } else if (lane == 0) {
        write_stat(a, which + 1, v, bad);
    }
}

// ---------------------------------------------------------------- two launches
// Each sequence's weight (seq_mean), or the active tokens in each block's share of the sequences
// (token_mean); and the main kernel's ticket set to 0.  Long sequences are counted by a cluster
// each.
__global__ void __launch_bounds__(1024) k_policy_count(const PolicyCall a) {
    __shared__ int smem[32];
    __shared__ int counted;
    cg::cluster_group cluster = cg::this_cluster();
    const int size = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int threads = blockDim.x;
    ptx::grid_dependents_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    const bool per_seq = a.reduction == RLK_REDUCE_SEQ_MEAN;
    if (a.reduction == RLK_REDUCE_SUM || (!per_seq && !a.active)) return;
    const int rows = per_seq ? a.n_seqs : kPolicyCountBlocks;
    for (int s = blockIdx.x / size; s < rows; s += gridDim.x / size) {
        int64_t b = 0, e = a.T;
        Bounds bd = {0, a.T};
        if (!per_seq) {
            // shares of the whole batch, so that the mask need not wait for the offsets
            const int64_t share = ((static_cast<int64_t>(a.T) + kPolicyCountBlocks - 1) / kPolicyCountBlocks + 15) / 16 * 16;
            bd = bounds_of(a);
            b = s * share;
            e = b + share < a.T ? b + share : a.T;
        } else if (a.offsets) {
            b = a.offsets[s];
            e = a.offsets[s + 1];
        }
        int n = static_cast<int>(e - b);
        if (a.active) {
            const int who = rank * threads + threadIdx.x, all = size * threads;
            n = count_active(a.active, b, e, a.T, who, all);
            if (!per_seq && (b < bd.first || e > bd.last))  // some lie outside all sequences
                n = count_active(a.active, b > bd.first ? b : bd.first, e < bd.last ? e : bd.last, a.T, who, all);
            n = __reduce_add_sync(0xffffffffu, n);
            if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = n;
            __syncthreads();
            n = 0;
            for (int i = 0; i < threads / 32; ++i) n += smem[i];
            if (size > 1) {
                if (threadIdx.x == 0) counted = n;
                cluster.sync();
                if (rank == 0 && threadIdx.x == 0) {
                    for (int c = 1; c < size; ++c) n += *cluster.map_shared_rank(&counted, c);
                }
                cluster.sync();
            } else {
                __syncthreads();
            }
        }
        if (rank == 0 && threadIdx.x == 0) {
            if (per_seq) a.weights[s] = seq_weight(a, n);
            else a.counts[s] = n;
        }
    }
}

template <int kKl>
__global__ void __launch_bounds__(kThreads, kMainCtasPerSm) k_policy_main(const PolicyCall a) {
    constexpr int kPer = kPolicyUnit / kThreads;
    __shared__ float4 spans[2][kUnitWarps];
    __shared__ float2 finish[kThreads / 32][4];
    __shared__ bool last_here;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    const int at = threadIdx.x * kPer;
    // offsets that descend or leave [0, T]: a share of them per CTA
    bool bad = false;
    if (a.offsets) {
        for (int64_t s = blockIdx.x + static_cast<int64_t>(threadIdx.x) * gridDim.x; s <= a.n_seqs;
             s += static_cast<int64_t>(kThreads) * gridDim.x) {
            const int b = a.offsets[s], e = s < a.n_seqs ? a.offsets[s + 1] : a.T;
            bad |= b < 0 || e < b || e > a.T;
        }
    }
    Tokens<kKl, kPer> k;
    k.load(a, blockIdx.x * static_cast<int64_t>(kPolicyUnit) + at);
    const Bounds bd = bounds_of(a);
    const bool by_mean = a.reduction == RLK_REDUCE_SEQ_MEAN;
    const bool by_seq = a.offsets && (a.adv_per_seq || by_mean);
    ptx::grid_dependency_wait();
    int n_all = bd.last - bd.first;
    if (a.active && a.reduction == RLK_REDUCE_TOKEN_MEAN) {
        static_assert(kPolicyCountBlocks == 256, "two int4 a lane");
        const int4 c0 = reinterpret_cast<const int4*>(a.counts)[lane];
        const int4 c1 = reinterpret_cast<const int4*>(a.counts)[lane + 32];
        n_all = __reduce_add_sync(0xffffffffu, c0.x + c0.y + c0.z + c0.w + c1.x + c1.y + c1.z + c1.w);
    }
    // a sequence mean over one sequence without offsets has one weight too
    const float w_all = by_mean && !a.offsets ? a.weights[0] : token_weight(a, n_all);
    int slot = 0;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        if (u != blockIdx.x) k.load(a, u * kPolicyUnit + at);
        k.cut(bd);
        float w[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) w[i] = w_all;
        const int64_t tf = k.t0 - lane * kPer, tl = tf + kPer * 32 - 1;
        if (by_seq && tf < a.T && a.n_seqs > 0) {
            const int last = static_cast<int>(tl < a.T ? tl : a.T - 1);
            const int lo = warp_find_seq(a.offsets, a.n_seqs, static_cast<int>(tf));
            if (lo + 1 >= a.n_seqs || a.offsets[lo + 1] > last) {
                // one sequence, as in most warps
                const float ws = by_mean ? a.weights[lo] : w_all;
                const float as = a.adv_per_seq ? a.advantages[lo] : 0.0f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    w[i] = ws;
                    if (a.adv_per_seq) k.adv[i] = as;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (!k.on[i]) continue;
                    const int s = find_seq(a.offsets, lo, a.n_seqs - 1, static_cast<int>(k.t0) + i);
                    if (by_mean) w[i] = a.weights[s];
                    if (a.adv_per_seq) k.adv[i] = a.advantages[s];
                }
            }
        }
        float4 terms[kPer];
        policy_tokens<kKl>(a, k, w, terms);
        const float4 s = span_sum(terms[0], terms[1], terms[2], terms[3]);
        if (lane == 0) spans[slot][warp] = s;
        bad = __syncthreads_or(bad);
        if (threadIdx.x < 4)
            reinterpret_cast<float*>(a.parts + u)[threadIdx.x] = bad ? CUDART_NAN_F : unit_sum(spans[slot], threadIdx.x);
        slot ^= 1;
    }
    // the last CTA to come here adds up the units; its tail is nobody's company, so it is kept short
    // (4.9 us at 1.77 M tokens with a fence by every thread, the offsets checked here, four loads at
    // a time and the stats one after the other)
    if (warp == 0) {
        __threadfence();
        __syncwarp();
        if (lane == 0) last_here = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) report_status(a.status, RLK_ERR_INVALID_ARG);
    if (!last_here) return;
    __threadfence();
    float2 v[4] = {};
    for (int64_t u0 = threadIdx.x; u0 < units; u0 += 8 * kThreads) {
        float4 p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            p[i] = u0 + i * kThreads < units ? __ldcg(a.parts + u0 + i * kThreads) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            two_add(v[0], p[i].x);
            two_add(v[1], p[i].y);
            two_add(v[2], p[i].z);
            two_add(v[3], p[i].w);
        }
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = pair_add(v[c], make_float2(__shfl_xor_sync(0xffffffffu, v[c].x, o),
                                              __shfl_xor_sync(0xffffffffu, v[c].y, o)));
    }
    if (lane < 4) finish[warp][lane] = lane == 0 ? v[0] : lane == 1 ? v[1] : lane == 2 ? v[2] : v[3];
    __syncthreads();
    if (warp != 0) return;
    // lane 8 c + w: stat c of warp w
    static_assert(kUnitWarps == 8, "eight lanes a stat");
    float2 s = finish[lane & 7][lane >> 3];
#pragma unroll 1
    for (int o = 4; o >= 1; o >>= 1)
        s = pair_add(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
    const float2 kl = make_float2(__shfl_sync(0xffffffffu, s.x, 8), __shfl_sync(0xffffffffu, s.y, 8));
    if ((lane & 7) == 0) write_stat(a, lane >> 3, s, bad);
    if (lane == 0) write_loss(a, s, kl, bad);
}

// Mean length from which a sequence is counted by a cluster of 8 CTAs of 1024 threads instead of
// one CTA of 256.  A sequence mean's whole call: 26.1 against 24.4 us at 49152 tokens each, 22.0
// against 22.7 at 58982 (1.77 M tokens in all); 10.5 against 10.3 at 32768, 10.3 against 12.3 at
// 65536 (262144 in all); 20.9 against 123 for one sequence of 1.77 M.  The lengths themselves are
// on the device: one long sequence among many short ones is counted by one CTA.
constexpr int kClusterCountTokens = 49152;

template <int kKl, int kCtas, int kPer>
cudaError_t launch_one(const PolicyCall& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.gridDim = dim3(kCtas, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCtas > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_policy_one<kKl, kCtas, kPer>, a);
}

}  // namespace

// One cluster up to 32768 tokens: 7.5 us against 7.5 in two launches at 16384, 7.7 against 7.6 at
// 32768, and a launch and a workspace less for the host (17.5 against 23.0 us a call).
bool policy_one_launch(int64_t T, int64_t n_seqs) {
    return T <= kCluster * 1024 * 4 && n_seqs <= kLaunchSeqs;
}

template <int kKl>
cudaError_t launch_kl(const PolicyCall& a, int num_sms, cudaStream_t stream) {
    // one CTA 4.1 against the cluster's 4.9 us at 128 tokens, 4.3 against 5.2 at 1024 (with four
    // tokens a thread 6.2 against 5.3 at 1100); the cluster with one token a thread 5.3 against 7.0
    // with four at 1100, 5.6 against 7.7 at 8192, where its threads end
    if (policy_one_launch(a.T, a.n_seqs))
        return a.T <= 1024              ? launch_one<kKl, 1, 1>(a, stream)
               : a.T <= kCluster * 1024 ? launch_one<kKl, kCluster, 1>(a, stream)
                                        : launch_one<kKl, kCluster, 4>(a, stream);
    int rows = 1;
    if (a.reduction == RLK_REDUCE_SEQ_MEAN) rows = a.n_seqs;
    else if (a.active && a.reduction == RLK_REDUCE_TOKEN_MEAN) rows = kPolicyCountBlocks;
    const int most = num_sms * 8;
    if (rows > most) rows = most;
    const bool lengthy = a.active && a.reduction == RLK_REDUCE_SEQ_MEAN && a.n_seqs > 0 && a.T / a.n_seqs > kClusterCountTokens;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    const int size = lengthy ? kCluster : 1;
    cfg.gridDim = dim3(static_cast<unsigned>((rows > 0 ? rows : 1) * size), 1, 1);
    cfg.blockDim = dim3(lengthy ? 1024 : a.reduction == RLK_REDUCE_TOKEN_MEAN ? 512 : kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_policy_count, a);
    if (e != cudaSuccess) return e;
    const int64_t units = (static_cast<int64_t>(a.T) + kPolicyUnit - 1) / kPolicyUnit;
    const int64_t resident = static_cast<int64_t>(num_sms) * kMainCtasPerSm;
    const int64_t ctas = units < resident ? units : resident;
    cfg.gridDim = dim3(static_cast<unsigned>(ctas > 0 ? ctas : 1), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_policy_main<kKl>, a);
}

cudaError_t launch_policy_loss(const PolicyArgs& args, int num_sms, cudaStream_t stream) {
    PolicyCall a;
    static_cast<PolicyArgs&>(a) = args;
    a.scale2 = split_two(a.scale);
    a.coef2 = split_two(a.kl_coef64);
    auto places = [](const void* p) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15); };
    a.wide = ((places(a.logprob) | places(a.old_logprob) | places(a.ref_logprob) | places(a.grad) |
               (a.adv_per_seq ? 0u : places(a.advantages)) | (places(a.active) & 3)) == 0);
    if (!a.ref_logprob) return launch_kl<0>(a, num_sms, stream);
    return a.kl_kind == RLK_KL_K1   ? launch_kl<RLK_KL_K1>(a, num_sms, stream)
           : a.kl_kind == RLK_KL_K2 ? launch_kl<RLK_KL_K2>(a, num_sms, stream)
                                    : launch_kl<RLK_KL_K3>(a, num_sms, stream);
}

}  // namespace rlk
