// Shared by the training-step operators (policy loss, preference loss,
// gradient clipping, RMSNorm backward): the launch interface between the host
// dispatcher and their kernels, and the device arithmetic they have in common.
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/rlk.h"
#include "rlk_contract.cuh"

namespace rlk {

// ---------------------------------------------------------------- launches
struct PolicyArgs {
    const float* logprob;     // [T]
    const float* old_logprob; // [T]
    const float* ref_logprob; // [T] or nullptr
    const float* advantages;  // [T], or [n_seqs] when adv_per_seq
    const uint8_t* active;    // [T] or nullptr
    const int32_t* offsets;   // [n_seqs + 1] or nullptr (one sequence [0, T))
    int T, n_seqs;
    int adv_per_seq;
    int kl_kind, reduction;
    // log(1 + clip_high), log(1 - clip_low), log(dual_clip), each as a sum of two floats
    float2 log_high, log_low, log_dual;
    float ratio_high, ratio_low, dual;  // 1 + clip_high, 1 - clip_low, dual_clip (0 = off)
    float kl_coef;
    double scale, kl_coef64;
    int32_t* ticket;          // workspace of the two-launch path: CTAs that are done
    int32_t* counts;          // workspace: active tokens per block (token_mean)
    float* weights;           // workspace: weight of each sequence's tokens (seq_mean)
    float4* parts;            // workspace: one (policy, kl, clipped, -d) sum per unit
    float* out_loss;          // [1]
    float* out_stats;         // [4]
    float* grad;              // [T] or nullptr
    int32_t* status;
};

constexpr int kPolicyUnit = 1024;         // tokens per partial sum
constexpr int kPolicyCountBlocks = 256;   // blocks counting a token mean's active tokens
// Whether a batch runs as one cluster, without a workspace.
bool policy_one_launch(int64_t T, int64_t n_seqs);
cudaError_t launch_policy_loss(const PolicyArgs& a, int num_sms, cudaStream_t stream);

struct PreferenceArgs {
    const float* logprob;     // [T]
    const float* ref_logprob; // [T] or nullptr
    const uint8_t* active;    // [T] or nullptr
    const int32_t* offsets;   // [2 * n_pairs + 1]
    int T, n_pairs;
    int halves;               // pair i = sequences (i, n_pairs + i), else (2i, 2i + 1)
    int kind, length_normalize;
    double beta, label_smoothing, margin;
    double half_over_beta;    // 1 / (2 beta)
    double scale_per_pair;    // scale / n_pairs
    float* out_loss;          // [1]
    float* out_pair_loss;     // [n_pairs]
    float* out_rewards;       // [2 * n_pairs], sequence order
    float* grad;              // [T] or nullptr
    // workspace of the path over all chunks
    int32_t* ticket;          // CTAs that are done
    float2* chunk_sums;       // as pairs
    int32_t* chunk_counts;
    int32_t* status;
};
// Largest batch that one cluster does alone: 9.2 us at one pair of 32768 tokens, where two
// launches take 9.6; at 65536 12.1 against 9.8.
constexpr int64_t kPreferenceClusterTokens = 32768;
// Tokens a pair from which the path over all chunks is taken.  Against a team of up to 8 CTAs a
// pair: 9.7 and 9.6 us at 32768 tokens, 9.6 and 11.1 at 50000, 9.9 and 15.7 at 100000 (one pair);
// 11.8 and 10.5, 11.9 and 12.1 at 32768 and 50000 (four pairs).
constexpr int64_t kPreferenceSplitTokens = 40960;
// Whether a batch takes the path over all chunks, and how many of them it has at most.
bool preference_split(int64_t T, int64_t n_pairs);
int64_t preference_chunks(int64_t T, int64_t n_pairs);
cudaError_t launch_preference_loss(const PreferenceArgs& a, int num_sms, cudaStream_t stream);

// Tensors of one launch: pointers and sizes travel by value in the kernel's parameters, so a
// captured launch holds them and nothing has to be copied to the device first.
struct ClipEntry {
    const void* in;
    void* out;
    int64_t n;
};
template <int kMost>
struct ClipTableOf {
    static constexpr int kSize = kMost;
    ClipEntry e[kMost];
    int32_t first[kMost + 1];  // each tensor's first piece within this launch
    uint8_t dtype[kMost];
    int count;
};
using ClipTable = ClipTableOf<640>;
using ClipTableSmall = ClipTableOf<64>;
struct ClipOut {
    float* norm;
    float* scale;             // nullptr: the norm alone is wanted
    int32_t* status;
    double max_norm;
};
constexpr int kClipPieceBytes = 16384;   // what a CTA works on at a time
constexpr int kClipCtasPerSm = 4;
constexpr int kClipSlots = 152 * kClipCtasPerSm;  // most CTAs of a launch, a partial sum each
// Largest set that one cluster does in one launch.  It saves the host a launch and a workspace,
// 20.4 against 27.3 us a call through Python at any of these sizes, and stays below that on the
// device, where two launches are faster from 12 pieces on: 7.2 against 4.6 us at 12 pieces in 12
// tensors, 12.1 against 4.7 at 48, 16.5 against 4.9 at 90 (3.7 against 4.2 at 2).
constexpr int kClipClusterPieces = 96;
// CTAs, and partial sums, of a launch over so many pieces.
inline int clip_launch_slots(int64_t pieces) { return pieces < kClipSlots ? static_cast<int>(pieces) : kClipSlots; }
cudaError_t launch_clip_cluster(const ClipTableSmall& t, const ClipOut& o, cudaStream_t stream);
// A launch's slots are pairs of floats.
cudaError_t launch_grad_sumsq(const ClipTable& t, float2* slots, cudaStream_t stream);
cudaError_t launch_grad_norm(const float2* slots, int n, const ClipOut& o, cudaStream_t stream);
// write: this launch stores norm and scale
cudaError_t launch_grad_scale(const ClipTable& t, const float2* slots, int n, const ClipOut& o,
                              bool write, cudaStream_t stream);

struct RmsBwdArgs {
    const void* grad_out;     // [T][H] fp32 or bf16
    const uint16_t* x;        // bf16 [T][H], the normalised rows' inputs
    const uint16_t* gamma;    // bf16 [H]
    const void* grad_res;     // [T][H] of grad_x's type, or nullptr
    void* grad_x;             // [T][H] fp32 or bf16
    float* grad_gamma;        // [H] or nullptr
    float* parts;             // workspace [blocks][H]
    float eps;
    int T, H;
    int go_dtype, gx_dtype;   // RLK_DTYPE_*
};
// Ranges of rows whose grad_gamma sums are formed apart, a CTA per SM each.
constexpr int kRmsBwdRanges = 152;
// Rows that one cluster of 8 CTAs takes alone, grad_gamma and all: a launch less for the host (13.4
// against 18.2 us a call at H = 4096) for little more time on the device (5.6 against 4.3 us at 16
// rows) as long as every team has one row; at 32 and 64 rows it would be 7.7 and 11.2 us against
// 4.7 and 4.9 for the two launches.
constexpr int64_t kRmsBwdClusterRows = 16;
inline bool rmsnorm_backward_one_launch(int64_t T) { return T > 0 && T <= kRmsBwdClusterRows; }
inline int rmsnorm_backward_ranges(int64_t T) { return T < kRmsBwdRanges ? static_cast<int>(T) : kRmsBwdRanges; }
cudaError_t launch_rmsnorm_backward(const RmsBwdArgs& a, cudaStream_t stream);

// A parameter as the sum of two floats (2^-48 relative), formed on the host: a conversion from fp64
// on the device is as slow as fp64 itself.
inline float2 split_two(double v) {
    const float hi = static_cast<float>(v);
    const float lo = std::isfinite(hi) ? static_cast<float>(v - static_cast<double>(hi)) : 0.0f;
    return make_float2(hi, lo);
}

// ---------------------------------------------------------------- device arithmetic
// a - b as the unevaluated sum of its rounded value and the rounding error, exactly
// (Moller-Knuth two-sum); the error is 0 where the difference is not finite.
__device__ __forceinline__ float2 two_diff(float a, float b) {
    const float s = __fsub_rn(a, b);
    const float t = __fsub_rn(s, a);
    const float e = __fsub_rn(__fsub_rn(a, __fsub_rn(s, t)), __fadd_rn(b, t));
    return make_float2(s, fabsf(s) < CUDART_INF_F ? e : 0.0f);
}

// (hi, lo) += x with the rounding error kept in lo.
__device__ __forceinline__ void two_add(float2& acc, float x) {
    const float s = __fadd_rn(acc.x, x);
    const float t = __fsub_rn(s, acc.x);
    const float e = __fadd_rn(__fsub_rn(acc.x, __fsub_rn(s, t)), __fsub_rn(x, t));
    acc.x = s;
    acc.y = __fadd_rn(acc.y, fabsf(s) < CUDART_INF_F ? e : 0.0f);
}

// Sum of two such pairs.  GB300 adds fp64 at a small fraction of the fp32 rate (a warp's fp64
// add takes tens of cycles of issue), so long sums are carried as pairs of floats, exact to about
// 2^-46 of the larger operand; a + b and b + a give the same bits.
__device__ __forceinline__ float2 pair_add(float2 a, float2 b) {
    const float s = __fadd_rn(a.x, b.x);
    const float t = __fsub_rn(s, a.x);
    const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
    const float lo = __fadd_rn(__fadd_rn(a.y, b.y), e);
    const float hi = __fadd_rn(s, lo);
    return fabsf(s) < CUDART_INF_F ? make_float2(hi, __fsub_rn(lo, __fsub_rn(hi, s))) : make_float2(s, 0.0f);
}
__device__ __forceinline__ float2 pair_of(float v) { return make_float2(v, 0.0f); }
__device__ __forceinline__ float2 pair_negated(float2 v) { return make_float2(-v.x, -v.y); }
// Product of two such pairs, to about 2^-45; its first part is the product rounded to fp32.
__device__ __forceinline__ float2 pair_mul(float2 a, float2 b) {
    const float p = __fmul_rn(a.x, b.x);
    const float e = __fmaf_rn(a.y, b.x, __fmaf_rn(a.x, b.y, __fmaf_rn(a.x, b.x, -p)));
    const float hi = __fadd_rn(p, e);
    return fabsf(p) < CUDART_INF_F ? make_float2(hi, __fsub_rn(e, __fsub_rn(hi, p))) : make_float2(p, 0.0f);
}
__device__ __forceinline__ float2 warp_sum(float2 v) {
    // not unrolled: a dependent chain either way, and small kernels pay for every line of code that
    // they fetch for the first time
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1)
        v = pair_add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}

__device__ __forceinline__ bool above(float2 d, float2 border) {
    return d.x > border.x || (d.x == border.x && d.y > border.y);
}

// exp over the whole fp32 range, NaN kept: the contract's reduction and polynomial (Cody-Waite,
// degree-7 Taylor), scaled by 2^n in two factors so that n = 128 and subnormal results are
// formed too; beyond the range the result is +inf or +0.
__device__ __forceinline__ float exp_any(float x) {
    const float xc = fminf(fmaxf(x, -104.0f), 89.0f);
    const float t = __fmaf_rn(xc, 0x1.715476p+0f, 0x1.8p+23f);
    const float n = __fsub_rn(t, 0x1.8p+23f);
    const int ni = __float_as_int(t) - __float_as_int(0x1.8p+23f);
    float r = __fmaf_rn(-n, 0x1.62e430p-1f, xc);
    r = __fmaf_rn(-n, -0x1.05c610p-29f, r);
    float p = 0x1.a01a02p-13f;
    p = __fmaf_rn(p, r, 0x1.6c16c2p-10f);
    p = __fmaf_rn(p, r, 0x1.111112p-7f);
    p = __fmaf_rn(p, r, 0x1.555556p-5f);
    p = __fmaf_rn(p, r, 0x1.555556p-3f);
    p = __fmaf_rn(p, r, 0.5f);
    p = __fmaf_rn(p, r, 1.0f);
    p = __fmaf_rn(p, r, 1.0f);
    const int half = ni >> 1;
    p = __fmul_rn(p, __int_as_float((half + 127) << 23));
    p = __fmul_rn(p, __int_as_float((ni - half + 127) << 23));
    return x != x ? x : p;
}

// e^u - 1 - u for |u| < 1, where that difference cancels: its Taylor series
// u^2 (1/2 + u/6 + ... + u^9/11!), the first term left out below 2^-27 of the sum.
constexpr int kExpTail = 10;
__device__ constexpr float exp_tail(int i) {  // 1/11! .. 1/2!
    constexpr float c[kExpTail] = {0x1.ae6456p-26f, 0x1.27e4fcp-22f, 0x1.71de3ap-19f, 0x1.a01a02p-16f,
                                   0x1.a01a02p-13f, 0x1.6c16c2p-10f, 0x1.111112p-7f,  0x1.555556p-5f,
                                   0x1.555556p-3f,  0.5f};
    return c[i];
}
// and for any u
__device__ __forceinline__ float exp_minus_1_minus(float u) {
    if (!(fabsf(u) < 1.0f)) return __fsub_rn(__fsub_rn(exp_any(u), 1.0f), u);
    float p = exp_tail(0);
#pragma unroll
    for (int i = 1; i < kExpTail; ++i) p = __fmaf_rn(p, u, exp_tail(i));
    return __fmul_rn(__fmul_rn(u, u), p);
}

// log(1 + e) for e in [0, 1]: 2 atanh(v), v = e / (2 + e) <= 1/3, by the odd series through
// v^17 (the next term is below 2^-32 of the sum).
__device__ __forceinline__ float log_1_plus(float e) {
    const float v = __fdiv_rn(e, __fadd_rn(2.0f, e));
    const float q = __fmul_rn(v, v);
    float p = 0x1.e1e1e2p-4f;              // 2/17
    p = __fmaf_rn(p, q, 0x1.111112p-3f);   // 2/15
    p = __fmaf_rn(p, q, 0x1.3b13b2p-3f);   // 2/13
    p = __fmaf_rn(p, q, 0x1.745d18p-3f);   // 2/11
    p = __fmaf_rn(p, q, 0x1.c71c72p-3f);   // 2/9
    p = __fmaf_rn(p, q, 0x1.24924ap-2f);   // 2/7
    p = __fmaf_rn(p, q, 0x1.99999ap-2f);   // 2/5
    p = __fmaf_rn(p, q, 0x1.555556p-1f);   // 2/3
    return __fmaf_rn(__fmul_rn(p, q), v, __fmul_rn(2.0f, v));
}

__device__ __forceinline__ void report_status(int32_t* status, int code) {
    if (status) atomicOr(status, 1 << code);
}

// The last s in [0, n) with offsets[s] <= t (0 where there is none), found by a whole warp in
// ceil(log32 n) dependent loads; every lane gets it.  With offsets that do not ascend the result
// is still in [0, n).
__device__ __forceinline__ int warp_find_seq(const int32_t* offsets, int n, int t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t p = lo + static_cast<int64_t>(lane) * step;
        const bool left = p < hi && (lane == 0 || offsets[p] <= t);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, left) | 1u);
        lo += k * step;
        hi = hi - lo < step ? hi : lo + step;
    }
    return lo;
}

// The same within [lo, hi], one thread alone.
__device__ __forceinline__ int find_seq(const int32_t* offsets, int lo, int hi, int t) {
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
}  // namespace rlk
