// Preference loss on paired log ratios, and its gradient with respect to the
// log-probabilities, for packed sequences.
//
//   m_q  = sum over sequence q's active tokens of (logprob - ref), divided by
//          their number with length_normalize (0 for a sequence without any)
//   h    = m_chosen - m_rejected,  z = beta h - margin
//   sigmoid  l = -(1 - eps) log sig(z) - eps log sig(-z),  dl/dh = beta (sig(z) - (1 - eps))
//   hinge    l = max(0, 1 - z),                            dl/dh = -beta where z < 1
//   ipo      l = (h - 1 / (2 beta))^2,                     dl/dh = 2 (h - 1 / (2 beta))
//   loss = scale mean_i l_i;  grad_t = +- scale / n_pairs dl/dh [/ active tokens]
//
// Order of a sequence's sum, the same wherever the sequence lies in the batch:
// tokens are counted from its first; a warp sums chunks of 256 of them (a
// lane takes every 32nd, compensated in fp32, then a shuffle tree in fp64);
// chunk g is added to slot g mod 1024 in ascending order, and the slots are
// added by a fixed tree in fp64.
#include "rlk_train.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 256;
constexpr int kSlots = 1024;

struct Span {
    int64_t b, e;
};

__device__ __forceinline__ Span span_of(const PreferenceArgs& a, int q) {
    Span s;
    s.b = a.offsets[q];
    s.e = a.offsets[q + 1];
    if (s.b < 0) s.b = 0;
    if (s.e > a.T) s.e = a.T;
    if (s.e < s.b) s.e = s.b;
    return s;
}

__device__ __forceinline__ double block_tree(const double* slots, double* tmp) {
    double v = 0.0;
    for (int i = threadIdx.x; i < kSlots; i += kThreads) v = __dadd_rn(v, slots[i]);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < kWarps; ++i) v = __dadd_rn(v, tmp[i]);
    __syncthreads();
    return v;
}

__device__ __forceinline__ void zero_range(float* grad, int64_t b, int64_t e) {
    for (int64_t t = b + threadIdx.x; t < e; t += kThreads) grad[t] = 0.0f;
}

__global__ void __launch_bounds__(kThreads) k_preference_pair(const PreferenceArgs a) {
    __shared__ double slots[2][kSlots];
    __shared__ int counts[2];
    __shared__ double tmp[kWarps];
    __shared__ float slope[2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pair = blockIdx.x;
    const int q[2] = {a.halves ? pair : 2 * pair, a.halves ? a.n_pairs + pair : 2 * pair + 1};
    for (int i = threadIdx.x; i < 2 * kSlots; i += kThreads) slots[i / kSlots][i % kSlots] = 0.0;
    if (threadIdx.x < 2) counts[threadIdx.x] = 0;
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const Span sp = span_of(a, q[side]);
        int n = 0;
        for (int64_t g = warp; sp.b + g * kChunk < sp.e; g += kWarps) {
            float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < kChunk / 32; ++i) {
                const int64_t t = sp.b + g * kChunk + i * 32 + lane;
                if (t >= sp.e || (a.active && a.active[t] == 0)) continue;
                ++n;
                const float2 d = two_diff(a.logprob[t], a.ref_logprob ? a.ref_logprob[t] : 0.0f);
                two_add(acc, d.x);
                acc.y = __fadd_rn(acc.y, d.y);
            }
            const double v = warp_sum(static_cast<double>(acc.x) + static_cast<double>(acc.y));
            if (lane == 0) slots[side][g % kSlots] += v;
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) atomicAdd(&counts[side], n);  // whole numbers: any order gives the same sum
    }
    __syncthreads();
    double m[2];
    m[0] = block_tree(slots[0], tmp);
    m[1] = block_tree(slots[1], tmp);
    if (threadIdx.x == 0) {
        double inv[2] = {1.0, 1.0};
        if (a.length_normalize) {
            for (int k = 0; k < 2; ++k) {
                inv[k] = 1.0 / (counts[k] > 1 ? counts[k] : 1);
                m[k] = m[k] * inv[k];
            }
        }
        const double h = m[0] - m[1];
        double loss, dh;
        if (a.kind == RLK_PREF_IPO) {
            const double off = h - 0.5 / a.beta;
            loss = off * off;
            dh = 2.0 * off;
        } else {
            const double zd = a.beta * h - a.margin;
            if (a.kind == RLK_PREF_HINGE) {
                loss = zd < 1.0 ? 1.0 - zd : (zd == zd ? 0.0 : zd);
                dh = zd < 1.0 ? -a.beta : (zd == zd ? 0.0 : zd);
            } else {
                // sig(z), sig(-z) and the two logs from e^-|z|, none of which cancels
                const float z = static_cast<float>(zd);
                const float e = exp_any(-fabsf(z));
                const double soft = static_cast<double>(log_1_plus(e));
                const double small = static_cast<double>(__fdiv_rn(e, __fadd_rn(1.0f, e)));  // sig(-|z|)
                const double pos = z >= 0.0f ? static_cast<double>(z) : 0.0;
                const double neg = z >= 0.0f ? 0.0 : -static_cast<double>(z);
                loss = (1.0 - a.label_smoothing) * (soft + neg) + a.label_smoothing * (soft + pos);
                // sig(z) - (1 - eps) = eps sig(z) - (1 - eps) sig(-z)
                const double sp = z >= 0.0f ? 1.0 - small : small, sn = z >= 0.0f ? small : 1.0 - small;
                dh = a.beta * (a.label_smoothing * sp - (1.0 - a.label_smoothing) * sn);
            }
        }
        a.out_pair_loss[pair] = static_cast<float>(loss);
        a.out_rewards[q[0]] = static_cast<float>(a.beta * m[0]);
        a.out_rewards[q[1]] = static_cast<float>(a.beta * m[1]);
        const double step = a.scale / a.n_pairs * dh;
        slope[0] = static_cast<float>(step * inv[0]);
        slope[1] = static_cast<float>(-step * inv[1]);
    }
    if (!a.grad) return;
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const Span sp = span_of(a, q[side]);
        const float g = slope[side];
        for (int64_t t = sp.b + threadIdx.x; t < sp.e; t += kThreads)
            a.grad[t] = (a.active && a.active[t] == 0) ? 0.0f : g;
    }
    // tokens before the first and behind the last sequence
    if (pair == 0) zero_range(a.grad, 0, span_of(a, 0).b);
    if (pair == a.n_pairs - 1) zero_range(a.grad, span_of(a, 2 * a.n_pairs - 1).e, a.T);
}

__global__ void __launch_bounds__(kThreads) k_preference_final(const PreferenceArgs a) {
    __shared__ double tmp[kWarps];
    bool bad = false;
    for (int s = threadIdx.x; s <= 2 * a.n_pairs; s += kThreads) {
        const int b = a.offsets[s], e = s < 2 * a.n_pairs ? a.offsets[s + 1] : a.T;
        bad |= b < 0 || e < b || e > a.T;
    }
    bad = __syncthreads_or(bad);
    double v = 0.0;
    for (int i = threadIdx.x; i < a.n_pairs; i += kThreads) v += static_cast<double>(a.out_pair_loss[i]);
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
        for (int i = 0; i < kWarps; ++i) v += tmp[i];
        if (a.n_pairs > 0) v = a.scale * (v / a.n_pairs);
        *a.out_loss = bad ? CUDART_NAN_F : static_cast<float>(v);
        if (bad) report_status(a.status, RLK_ERR_INVALID_ARG);
    }
}

}  // namespace

cudaError_t launch_preference_loss(const PreferenceArgs& a, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    if (a.n_pairs > 0) {
        k_preference_pair<<<a.n_pairs, kThreads, 0, stream>>>(a);
    } else if (a.grad && a.T > 0) {
        const cudaError_t e = cudaMemsetAsync(a.grad, 0, size_t(a.T) * sizeof(float), stream);
        if (e != cudaSuccess) return e;
    }
    k_preference_final<<<1, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace rlk
