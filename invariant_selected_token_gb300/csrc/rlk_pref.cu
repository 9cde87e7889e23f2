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
// Order of a sequence's sum, the same wherever the sequence lies in the batch
// and however many CTAs share it: tokens are counted from its first; a warp
// sums chunks of 256 of them (a lane takes every 32nd, compensated in fp32,
// then a shuffle tree in fp64); chunk g is added to slot g mod 1024 in
// ascending order, and the slots are added by a fixed tree in fp64.
//
// A pair is the work of a team of 1, 2, 4 or 8 CTAs of one cluster.  They
// meet in the shared memory of the team's first CTA: slots in, the two
// sequences' slopes out.  Small batches run as one cluster, which also adds
// up the pairs' losses; larger ones as a cluster per pair and a second launch
// for that sum.
#include <cooperative_groups.h>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 256;
constexpr int kSlots = 1024;
constexpr int kCluster = 8;

struct Span {
    int64_t b, e;
};

__device__ __forceinline__ Span span_of(const PreferenceArgs& a, int64_t q) {
    Span s;
    s.b = a.offsets[q];
    s.e = a.offsets[q + 1];
    if (s.b < 0) s.b = 0;
    if (s.e > a.T) s.e = a.T;
    if (s.e < s.b) s.e = s.b;
    return s;
}

// A pair's loss, rewards and slopes from its two sums and counts, by one thread.
__device__ __forceinline__ void pair_terms(const PreferenceArgs& a, int pair, int64_t q0, int64_t q1,
                                           double m0, double m1, int n0, int n1, float* slope) {
    double inv0 = 1.0, inv1 = 1.0;
    if (a.length_normalize) {
        inv0 = 1.0 / (n0 > 1 ? n0 : 1);
        inv1 = 1.0 / (n1 > 1 ? n1 : 1);
        m0 *= inv0;
        m1 *= inv1;
    }
    const double h = m0 - m1;
    double loss, dh;
    if (a.kind == RLK_PREF_IPO) {
        const double off = h - a.half_over_beta;
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
    a.out_rewards[q0] = static_cast<float>(a.beta * m0);
    a.out_rewards[q1] = static_cast<float>(a.beta * m1);
    const double step = a.scale_per_pair * dh;
    slope[0] = static_cast<float>(step * inv0);
    slope[1] = static_cast<float>(-step * inv1);
}

// The loss from the pairs' losses, by a whole CTA of kThreads.
__device__ __forceinline__ void preference_finish(const PreferenceArgs& a, double* tmp) {
    bool bad = false;
    const int64_t n = 2 * static_cast<int64_t>(a.n_pairs);
    for (int64_t s = threadIdx.x; s <= n; s += kThreads) {
        const int b = a.offsets[s], e = s < n ? a.offsets[s + 1] : a.T;
        bad |= b < 0 || e < b || e > a.T;
    }
    bad = __syncthreads_or(bad);
    double v = 0.0;
    for (int i = threadIdx.x; i < a.n_pairs; i += kThreads)
        v += static_cast<double>(__ldcg(a.out_pair_loss + i));
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        v = 0.0;
        for (int i = 0; i < kWarps; ++i) v += tmp[i];
        if (a.n_pairs > 0) v = a.scale_per_pair * v;
        *a.out_loss = bad ? CUDART_NAN_F : static_cast<float>(v);
        if (bad) report_status(a.status, RLK_ERR_INVALID_ARG);
    }
}

// One launch of clusters; every `team` CTAs of a cluster take a pair.
__global__ void __launch_bounds__(kThreads) k_preference(const PreferenceArgs a, int team, int finish) {
    __shared__ double slots[2][kSlots];
    __shared__ int counts[2];
    __shared__ double tmp[2][kWarps];
    __shared__ float slope[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int member = rank % team, lead = rank - member;
    const int teams = size / team;
    const int stride = gridDim.x / team;  // pairs in flight
    const int first = static_cast<int>(blockIdx.x) / size * teams + rank / team;
    double (*const lead_slots)[kSlots] =
        reinterpret_cast<double (*)[kSlots]>(cluster.map_shared_rank(&slots[0][0], lead));
    int* const lead_counts = cluster.map_shared_rank(counts, lead);
    const float* const lead_slope = cluster.map_shared_rank(slope, lead);
    const int rounds = (a.n_pairs + stride - 1) / stride;
    for (int r = 0; r < rounds; ++r) {
        const int pair = first + r * stride;
        const bool work = pair < a.n_pairs;
        const int64_t q[2] = {a.halves ? pair : 2 * static_cast<int64_t>(pair),
                              a.halves ? a.n_pairs + static_cast<int64_t>(pair) : 2 * static_cast<int64_t>(pair) + 1};
        Span sp[2] = {{0, 0}, {0, 0}};
        if (work) {
            sp[0] = span_of(a, q[0]);
            sp[1] = span_of(a, q[1]);
        }
        for (int i = threadIdx.x; i < 2 * kSlots; i += kThreads) slots[i / kSlots][i % kSlots] = 0.0;
        if (threadIdx.x < 2) counts[threadIdx.x] = 0;
        if (team > 1) cluster.sync(); else __syncthreads();
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            int n = 0;
            for (int64_t g = member * kWarps + warp; sp[side].b + g * kChunk < sp[side].e; g += team * kWarps) {
                float lp[kChunk / 32], ref[kChunk / 32];
                bool on[kChunk / 32];
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i) {
                    const int64_t t = sp[side].b + g * kChunk + i * 32 + lane;
                    const bool in = t < sp[side].e;
                    lp[i] = in ? a.logprob[t] : 0.0f;
                    ref[i] = in && a.ref_logprob ? a.ref_logprob[t] : 0.0f;
                    on[i] = in && (!a.active || a.active[t] != 0);
                }
                float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < kChunk / 32; ++i) {
                    if (!on[i]) continue;
                    ++n;
                    const float2 d = two_diff(lp[i], ref[i]);
                    two_add(acc, d.x);
                    acc.y = __fadd_rn(acc.y, d.y);
                }
                const double v = warp_sum(static_cast<double>(acc.x) + static_cast<double>(acc.y));
                if (lane == 0) {
                    // a slot is only ever this warp's
                    double* const slot = &lead_slots[side][g % kSlots];
                    *slot = __dadd_rn(*slot, v);
                }
            }
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0 && n) atomicAdd(&lead_counts[side], n);  // whole numbers: any order will do
        }
        if (team > 1) cluster.sync(); else __syncthreads();
        if (member == 0 && work) {
            double v[2];
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                v[side] = 0.0;
                for (int i = threadIdx.x; i < kSlots; i += kThreads) v[side] = __dadd_rn(v[side], slots[side][i]);
                v[side] = warp_sum(v[side]);
                if (lane == 0) tmp[side][warp] = v[side];
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                v[0] = v[1] = 0.0;
                for (int i = 0; i < kWarps; ++i) {
                    v[0] = __dadd_rn(v[0], tmp[0][i]);
                    v[1] = __dadd_rn(v[1], tmp[1][i]);
                }
                pair_terms(a, pair, q[0], q[1], v[0], v[1], counts[0], counts[1], slope);
            }
        }
        if (team > 1) cluster.sync(); else __syncthreads();
        if (a.grad && work) {
            const int who = member * kThreads + threadIdx.x, all = team * kThreads;
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const float g = lead_slope[side];
#pragma unroll 4
                for (int64_t t = sp[side].b + who; t < sp[side].e; t += all)
                    a.grad[t] = (a.active && a.active[t] == 0) ? 0.0f : g;
            }
            // tokens before the first and behind the last sequence
            if (pair == 0)
                for (int64_t t = who, e = span_of(a, 0).b; t < e; t += all) a.grad[t] = 0.0f;
            if (pair == a.n_pairs - 1)
                for (int64_t t = span_of(a, 2 * static_cast<int64_t>(a.n_pairs) - 1).e + who; t < a.T; t += all)
                    a.grad[t] = 0.0f;
        }
        __syncthreads();  // slots, counts and slopes are free for the next round
    }
    // nobody leaves while its shared memory may be read; the pairs' losses are out
    if (finish) __threadfence();
    cluster.sync();
    if (finish && rank == 0) {
        if (finish) __threadfence();
        preference_finish(a, tmp[0]);
    }
}

__global__ void __launch_bounds__(kThreads) k_preference_final(const PreferenceArgs a) {
    __shared__ double tmp[kWarps];
    ptx::grid_dependency_wait();
    preference_finish(a, tmp);
}

}  // namespace

cudaError_t launch_preference_loss(const PreferenceArgs& a, int num_sms, cudaStream_t stream) {
    if (a.n_pairs == 0 && a.grad && a.T > 0) {
        const cudaError_t e = cudaMemsetAsync(a.grad, 0, size_t(a.T) * sizeof(float), stream);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    const int64_t mean = a.n_pairs ? a.T / a.n_pairs : 0;  // tokens of a pair, about
    if (a.T <= kPreferenceClusterTokens || a.n_pairs == 0) {
        // teams so large that the cluster's CTAs all have a pair
        int team = kCluster;
        while (team > 1 && kCluster / team < a.n_pairs) team /= 2;
        cfg.gridDim = dim3(kCluster, 1, 1);
        attr[0].val.clusterDim.x = kCluster;
        return cudaLaunchKernelEx(&cfg, k_preference, a, team, 1);
    }
    // CTAs per pair: enough to fill the device, and none with less than 4096 tokens
    int team = 1;
    while (team < kCluster && static_cast<int64_t>(a.n_pairs) * team < num_sms * 2 && mean / (2 * team) >= 4096) team *= 2;
    const int64_t most = static_cast<int64_t>(num_sms) * 16 / team;
    const int64_t clusters = a.n_pairs < most ? a.n_pairs : most;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * team), 1, 1);
    attr[0].val.clusterDim.x = team;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k_preference, a, team, 0);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(1, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, k_preference_final, a);
}

}  // namespace rlk
