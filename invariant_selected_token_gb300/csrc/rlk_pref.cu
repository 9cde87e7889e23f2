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
// sums chunks of 256 of them (a lane takes every 32nd, then a shuffle tree);
// chunk g is added to slot g mod 1024 in ascending order, and the slots are
// added by a fixed tree.  All sums are pairs of floats.
//
// Up to 8 pairs of up to kPreferenceClusterTokens tokens in all run as one
// cluster in one launch: a pair is the work of a team of 1, 2, 4 or 8 of its
// CTAs, which meet in the shared memory of the team's first one (slots in, the
// two sequences' slopes out), and the first CTA adds up the pairs' losses.
// More pairs or tokens run the same kernel with a team per pair and add up in
// a second launch.  A few very long pairs, whose teams would leave most of the
// device idle, take one launch over all chunks and one over all tokens, whose
// CTAs each form the slopes they need.
//
// What bounds it: latency.  5.4 us a call on the device for 4 pairs of 255
// tokens, 7.7 for 64 pairs of 2048 (1.7 MB), 14.5 for 4 pairs of 262144 (13.6
// MB, 2.0 us of HBM): a launch, the offsets, the tokens, three barriers and a
// pair's terms one after the other.  With fp64 sums over the tokens the three
// took 14, 14 and 43 us; with the rejected sequence's tokens read after the
// chosen one's 7.5, 10.4 and 17.1; with a pair's terms in fp64 5.8, 8.1 and
// 15.1.
#include <cooperative_groups.h>
#include <limits>

#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;            // of a CTA; 128 for short pairs
constexpr int kWarps = kThreads / 32;    // warps of the sums' order, whatever the CTA has
constexpr int kChunk = 256;
constexpr int kSlots = 1024;
constexpr int kCluster = 8;

struct PreferenceCall : PreferenceArgs {
    float smooth32, keep32;                       // label_smoothing and 1 - it
    float2 beta2, margin2, half_over_beta2, scale2;  // the last one scale / n_pairs
};

struct Span {
    int64_t b, e;
};

__device__ __forceinline__ Span span_of(const PreferenceCall& a, int64_t q) {
    Span s;
    s.b = a.offsets[q];
    s.e = a.offsets[q + 1];
    if (s.b < 0) s.b = 0;
    if (s.b > a.T) s.b = a.T;
    if (s.e > a.T) s.e = a.T;
    if (s.e < s.b) s.e = s.b;
    return s;
}

// A sequence's mean from its sum, and 1 / (its active tokens).
__device__ __forceinline__ float2 mean_of(float2 sum, int n, float& inv) {
    const int c = n > 1 ? n : 1;
    const float hi = static_cast<float>(c), lo = static_cast<float>(c - static_cast<int64_t>(hi));
    inv = __fdiv_rn(1.0f, hi);
    // a quotient within a few steps, and the remainder's
    const float q = __fmul_rn(sum.x, inv);
    const float r = __fmaf_rn(-q, lo, __fadd_rn(__fmaf_rn(-q, hi, sum.x), sum.y));
    const float e = __fmul_rn(r, inv), m = __fadd_rn(q, e);
    return fabsf(q) < CUDART_INF_F ? make_float2(m, __fsub_rn(e, __fsub_rn(m, q))) : pair_of(q);
}

// A pair's loss, rewards and slopes from its two sums and counts, by two lanes, each of which
// writes one of the rewards.  What cancels (the two sums, z, the distance from 1 / (2 beta)) is
// formed as pairs of floats, the rest in fp32; in fp64 it took 1 us, one operation after another.
__device__ __forceinline__ void pair_terms(const PreferenceCall& a, int pair, int64_t q0, int64_t q1,
                                           float2 s0, float2 s1, int n0, int n1, bool write,
                                           float* slope, float* held_loss) {
    float2 m0 = s0, m1 = s1;
    float inv0 = 1.0f, inv1 = 1.0f;
    if (a.length_normalize) {
        m0 = mean_of(s0, n0, inv0);
        m1 = mean_of(s1, n1, inv1);
    }
    const float2 h = pair_add(m0, pair_negated(m1));
    const float beta = a.beta2.x;
    float loss, dh;
    if (a.kind == RLK_PREF_IPO) {
        const float off = pair_add(h, pair_negated(a.half_over_beta2)).x;
        loss = __fmul_rn(off, off);
        dh = __fmul_rn(2.0f, off);
    } else if (a.kind == RLK_PREF_HINGE) {
        // whether z < 1 is a decision, on sums that may well be whole numbers: beta itself, in fp64
        const double z = __fma_rn(a.beta, __dadd_rn(static_cast<double>(h.x), static_cast<double>(h.y)), -a.margin);
        const float gap = static_cast<float>(__dsub_rn(1.0, z));
        loss = gap > 0.0f ? gap : (gap == gap ? 0.0f : gap);
        dh = z < 1.0 ? -beta : (z == z ? 0.0f : gap);
    } else {
        // sig(z), sig(-z) and the two logs from e^-|z|, none of which cancels
        const float z = pair_add(pair_mul(a.beta2, h), pair_negated(a.margin2)).x;
        const float eps = a.smooth32, keep = a.keep32;
        const float e = exp_any(-fabsf(z));
        const float soft = log_1_plus(e);
        const float small = __fdiv_rn(e, __fadd_rn(1.0f, e));  // sig(-|z|)
        const float large = __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
        const float near = soft, far = __fadd_rn(soft, fabsf(z));  // -log sig(|z|), -log sig(-|z|)
        const bool up = z >= 0.0f;
        // a part with weight 0 is 0 even where its log is infinite
        loss = __fadd_rn(keep != 0.0f ? __fmul_rn(keep, up ? near : far) : 0.0f,
                         eps != 0.0f ? __fmul_rn(eps, up ? far : near) : 0.0f);
        if (z != z) loss = z;
        // sig(z) - (1 - eps) = eps sig(z) - (1 - eps) sig(-z)
        dh = __fmul_rn(beta, __fsub_rn(__fmul_rn(eps, up ? large : small), __fmul_rn(keep, up ? small : large)));
    }
    const int lane = threadIdx.x & 31;
    if (write) a.out_rewards[lane == 0 ? q0 : q1] = pair_mul(a.beta2, lane == 0 ? m0 : m1).x;
    if (lane != 0) return;
    if (write) a.out_pair_loss[pair] = loss;
    if (held_loss) *held_loss = loss;
    const float step = __fmul_rn(a.scale2.x, dh);
    slope[0] = __fmul_rn(step, inv0);
    slope[1] = -__fmul_rn(step, inv1);
}

__device__ __forceinline__ int64_t chosen_of(const PreferenceCall& a, int pair) {
    return a.halves ? pair : 2 * static_cast<int64_t>(pair);
}
__device__ __forceinline__ int64_t rejected_of(const PreferenceCall& a, int pair) {
    return a.halves ? a.n_pairs + static_cast<int64_t>(pair) : 2 * static_cast<int64_t>(pair) + 1;
}

// Offsets that descend or leave [0, T], as far as this thread sees.
__device__ __forceinline__ bool offsets_bad(const PreferenceCall& a) {
    bool bad = false;
    const int64_t n = 2 * static_cast<int64_t>(a.n_pairs);
    for (int64_t s = threadIdx.x; s <= n; s += blockDim.x) {
        const int b = a.offsets[s], e = s < n ? a.offsets[s + 1] : a.T;
        bad |= b < 0 || e < b || e > a.T;
    }
    return bad;
}

// The loss from the pairs' losses, by a whole CTA.
__device__ __forceinline__ void preference_finish(const PreferenceCall& a, const float* losses, bool bad, float2* tmp) {
    bad = __syncthreads_or(bad);
    auto finish = [&](float2 v) {
        if (threadIdx.x != 0) return;
        *a.out_loss = bad ? CUDART_NAN_F : pair_mul(a.scale2, v).x;
        if (bad) report_status(a.status, RLK_ERR_INVALID_ARG);
    };
    // warp w of 16 takes losses 32 w + lane, + 512, ...; those without any would add zeros
    if (a.n_pairs <= 32) {
        const int i = threadIdx.x;
        if (i < 32) finish(warp_sum(pair_of(i < a.n_pairs ? losses[i] : 0.0f)));
        return;
    }
    for (int w = threadIdx.x >> 5; w < kWarps && w * 32 < a.n_pairs; w += blockDim.x >> 5) {
        float2 v = pair_of(0.0f);
        for (int i = w * 32 + (threadIdx.x & 31); i < a.n_pairs; i += kThreads) v = pair_add(v, pair_of(losses[i]));
        v = warp_sum(v);
        if ((threadIdx.x & 31) == 0) tmp[w] = v;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int w = threadIdx.x;
        finish(warp_sum(w < kWarps && w * 32 < a.n_pairs ? tmp[w] : pair_of(0.0f)));
    }
}

// Sum and active tokens of chunk g of a sequence, by a warp, on every lane.
__device__ __forceinline__ float2 chunk_sum(const PreferenceCall& a, const Span& sp, int64_t g, int* count) {
    const int lane = threadIdx.x & 31;
    float lp[kChunk / 32], ref[kChunk / 32];
    bool on[kChunk / 32];
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) {
        const int64_t t = sp.b + g * kChunk + i * 32 + lane;
        const bool in = t < sp.e;
        lp[i] = in ? a.logprob[t] : 0.0f;
        ref[i] = in && a.ref_logprob ? a.ref_logprob[t] : 0.0f;
        on[i] = in && (!a.active || a.active[t] != 0);
    }
    float2 acc = pair_of(0.0f);
    int n = 0;
#pragma unroll
    for (int i = 0; i < kChunk / 32; ++i) {
        n += on[i];
        const float2 d = two_diff(on[i] ? lp[i] : 0.0f, on[i] ? ref[i] : 0.0f);
        two_add(acc, d.x);
        acc.y = __fadd_rn(acc.y, d.y);
    }
    *count = __reduce_add_sync(0xffffffffu, n);
    return warp_sum(pair_add(acc, pair_of(0.0f)));
}

__device__ __forceinline__ int64_t chunks_of(const Span& s) { return (s.e - s.b + kChunk - 1) / kChunk; }

struct PairScratch {
    float2 tmp[2][kWarps];
    int n[2][kWarps];
};

// Slots of both sequences -> the pair's terms, by a whole CTA; `slope` and the outputs are set
// by thread 0, so a barrier has to follow.  slot(side, j, n) gives a slot's sum and its active
// tokens; slots from chunks_of() on are empty.
template <typename SlotOf>
__device__ __forceinline__ void reduce_pair(const PreferenceCall& a, int pair, const Span (&sp)[2], SlotOf slot,
                                            bool write, PairScratch& sc, float* slope, float* held_loss) {
    const int lane = threadIdx.x & 31;
    int held[2];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int64_t c = chunks_of(sp[side]);
        held[side] = c < kSlots ? static_cast<int>(c) : kSlots;
    }
    // warp w of 16 takes slots 32 w + lane and + 512; those without any would add zeros
    const int most = held[0] > held[1] ? held[0] : held[1];
    for (int w = threadIdx.x >> 5; w < kWarps && w * 32 < most; w += blockDim.x >> 5) {
        float2 v[2][2];
        int n[2][2];
#pragma unroll
        for (int side = 0; side < 2; ++side) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = w * 32 + lane + k * kThreads;
                v[side][k] = pair_of(0.0f);
                n[side][k] = 0;
                if (i < held[side]) v[side][k] = slot(side, i, n[side][k]);
            }
        }
        float2 sum[2] = {pair_add(v[0][0], v[0][1]), pair_add(v[1][0], v[1][1])};
#pragma unroll 1
        for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
            for (int side = 0; side < 2; ++side)
                sum[side] = pair_add(sum[side], make_float2(__shfl_xor_sync(0xffffffffu, sum[side].x, o),
                                                            __shfl_xor_sync(0xffffffffu, sum[side].y, o)));
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int count = __reduce_add_sync(0xffffffffu, n[side][0] + n[side][1]);
            if (lane == 0) {
                sc.tmp[side][w] = sum[side];
                sc.n[side][w] = count;
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        // lanes 0 .. 15 add the chosen side's warps, lanes 16 .. 31 the rejected one's
        const int side = lane >> 4, w = lane & 15;
        const bool have = w * 32 < (side ? held[1] : held[0]);
        float2 v = have ? sc.tmp[side][w] : pair_of(0.0f);
        int n = have ? sc.n[side][w] : 0;
#pragma unroll 1
        for (int o = 8; o >= 1; o >>= 1) {
            v = pair_add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        const float2 v1 = make_float2(__shfl_sync(0xffffffffu, v.x, 16), __shfl_sync(0xffffffffu, v.y, 16));
        const int n1 = __shfl_sync(0xffffffffu, n, 16);
        if (lane < 2)
            pair_terms(a, pair, chosen_of(a, pair), rejected_of(a, pair), v, v1, n, n1, write, slope, held_loss);
    }
}

// ---------------------------------------------------------------- a team of CTAs per pair
// One launch of clusters; every `team` CTAs of a cluster take a pair at a time.  alone: this is
// the only cluster, and it also forms the loss.
__global__ void __launch_bounds__(kThreads, 2) k_preference(const PreferenceCall a, int team, int alone) {
    __shared__ float2 slots[2][kSlots];
    __shared__ int counts[2][kSlots];
    __shared__ PairScratch scratch;
    __shared__ float slope[2];
    __shared__ float losses[kCluster];  // the first CTA's, when alone
    cg::cluster_group cluster = cg::this_cluster();
    ptx::grid_dependents_launch();
    cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank()), size = static_cast<int>(cluster.num_blocks());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int member = rank % team, lead = rank - member;
    const int teams = size / team;
    const int stride = gridDim.x / team;  // pairs in flight
    const int first = static_cast<int>(blockIdx.x) / size * teams + rank / team;
    float2* const lead_slots = cluster.map_shared_rank(&slots[0][0], lead);
    int* const lead_counts = cluster.map_shared_rank(&counts[0][0], lead);
    const float* const lead_slope = cluster.map_shared_rank(slope, lead);
    float* const all_losses = cluster.map_shared_rank(losses, 0);
    const bool bad = alone && rank == 0 ? offsets_bad(a) : false;
    cluster.barrier_wait();  // every CTA has started: its shared memory may be written
    const int rounds = (a.n_pairs + stride - 1) / stride;
    for (int r = 0; r < rounds; ++r) {
        const int pair = first + r * stride;
        const bool work = pair < a.n_pairs;
        Span sp[2] = {{0, 0}, {0, 0}};
        if (work) {
            sp[0] = span_of(a, chosen_of(a, pair));
            sp[1] = span_of(a, rejected_of(a, pair));
        }
        // the two sequences' chunks one after the other
        const int64_t c0 = chunks_of(sp[0]), c01 = c0 + chunks_of(sp[1]);
        for (int64_t j = member * warps + warp; j < c01; j += team * warps) {
            const int side = j >= c0;
            const int64_t g = side ? j - c0 : j;
            int n;
            const float2 v = chunk_sum(a, side ? sp[1] : sp[0], g, &n);
            if (lane == 0) {
                // a slot is only ever this warp's: the warps of a team are a power of two
                const int at = side * kSlots + static_cast<int>(g % kSlots);
                lead_slots[at] = g < kSlots ? v : pair_add(lead_slots[at], v);
                lead_counts[at] = (g < kSlots ? 0 : lead_counts[at]) + n;
            }
        }
        if (team > 1) cluster.sync(); else __syncthreads();
        if (member == 0 && work)
            reduce_pair(a, pair, sp,
                        [&](int side, int j, int& n) {
                            n = counts[side][j];
                            return slots[side][j];
                        },
                        true, scratch, slope, alone ? all_losses + pair : nullptr);
        if (team > 1) cluster.sync(); else __syncthreads();
        if (a.grad && work) {
            const int who = member * blockDim.x + threadIdx.x, all = team * blockDim.x;
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
        // slots and slope are written again only behind a barrier that everyone reaches after
        // reading them: with one CTA per team that is this one
        if (team == 1) __syncthreads();
    }
    cluster.sync();  // nobody leaves while its shared memory may be read; all losses are there
    if (alone && rank == 0) preference_finish(a, losses, bad, scratch.tmp[0]);
}

__global__ void __launch_bounds__(kThreads) k_preference_final(const PreferenceCall a) {
    __shared__ float2 tmp[kWarps];
    const bool bad = offsets_bad(a);
    ptx::grid_dependency_wait();
    preference_finish(a, a.out_pair_loss, bad, tmp);
}

// ---------------------------------------------------------------- all CTAs over all pairs
constexpr int kSplitSeqs = 64;  // most sequences of this path: two a lane

// Each sequence's tokens and first chunk in the launches' common numbering, held by the lanes of
// every warp, so that nothing but the offsets is waited for; no chunk at all where the offsets
// descend (the numbering would outgrow the workspace).
struct ChunkMap {
    Span span[2];  // of sequences 2 lane and 2 lane + 1
    int first[2], total;
    bool bad;
    __device__ __forceinline__ void build(const PreferenceCall& a) {
        const int lane = threadIdx.x & 31, n = 2 * a.n_pairs;
        int o[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) o[k] = a.offsets[2 * lane + k < n ? 2 * lane + k : n];
        bad = __any_sync(0xffffffffu, o[0] < 0 || o[1] < o[0] || o[2] < o[1] || o[2] > a.T);
        int c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            span[k].b = bad ? 0 : o[k];
            span[k].e = bad ? 0 : o[k + 1];
            c[k] = static_cast<int>(chunks_of(span[k]));
        }
        int v = c[0] + c[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        first[0] = v - c[0] - c[1];
        first[1] = v - c[1];
        total = __shfl_sync(0xffffffffu, v, 31);
    }
    // The rest by whole warps.  The sequence that holds chunk i < total (empty ones hold none):
    __device__ __forceinline__ int seq_of(int i) const {
        const unsigned m0 = __ballot_sync(0xffffffffu, first[0] <= i), m1 = __ballot_sync(0xffffffffu, first[1] <= i);
        const int k0 = 31 - __clz(m0), k1 = 31 - __clz(m1);  // m0 has lane 0; an empty m1 gives -1
        return k1 >= k0 ? 2 * k1 + 1 : 2 * k0;
    }
    __device__ __forceinline__ int first_of(int q) const {
        return __shfl_sync(0xffffffffu, q & 1 ? first[1] : first[0], q >> 1);
    }
    __device__ __forceinline__ Span span_at(int q) const {
        Span s;
        s.b = __shfl_sync(0xffffffffu, static_cast<int>(q & 1 ? span[1].b : span[0].b), q >> 1);
        s.e = __shfl_sync(0xffffffffu, static_cast<int>(q & 1 ? span[1].e : span[0].e), q >> 1);
        return s;
    }
};

__global__ void __launch_bounds__(kThreads) k_preference_chunks(const PreferenceCall a) {
    ptx::grid_dependents_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    ChunkMap map;
    map.build(a);
    for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < map.total; i += gridDim.x * kWarps) {
        const int q = map.seq_of(i);
        int n;
        const float2 v = chunk_sum(a, map.span_at(q), i - map.first_of(q), &n);
        if ((threadIdx.x & 31) == 0) {
            a.chunk_sums[i] = v;
            a.chunk_counts[i] = n;
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_preference_spread(const PreferenceCall a) {
    __shared__ PairScratch scratch;
    __shared__ float slope[2];
    __shared__ bool last_here;
    ChunkMap map;
    map.build(a);
    ptx::grid_dependency_wait();
    auto slopes_of = [&](int pair, bool write) {
        const int q0 = static_cast<int>(chosen_of(a, pair)), q1 = static_cast<int>(rejected_of(a, pair));
        const Span sp[2] = {map.span_at(q0), map.span_at(q1)};
        const int at[2] = {map.first_of(q0), map.first_of(q1)};
        __syncthreads();  // the previous pair's slopes have been read
        reduce_pair(a, pair, sp,
                    [&](int side, int j, int& n) {
                        float2 v = a.chunk_sums[at[side] + j];
                        n = a.chunk_counts[at[side] + j];
                        for (int64_t g = j + kSlots, c = chunks_of(sp[side]); g < c; g += kSlots) {
                            v = pair_add(v, a.chunk_sums[at[side] + g]);
                            n += a.chunk_counts[at[side] + g];
                        }
                        return v;
                    },
                    write, scratch, slope, nullptr);
        __syncthreads();
    };
    // a pair's own outputs are written by the CTA that has its chosen sequence's first chunk, or,
    // where that sequence is empty, by CTA pair mod grid
    int have = -1;
    for (int pair = blockIdx.x; pair < a.n_pairs; pair += gridDim.x) {
        if (chunks_of(map.span_at(static_cast<int>(chosen_of(a, pair)))) > 0) continue;
        slopes_of(pair, true);
        have = pair;
    }
    const int i0 = static_cast<int>(static_cast<int64_t>(map.total) * blockIdx.x / gridDim.x);
    const int i1 = static_cast<int>(static_cast<int64_t>(map.total) * (blockIdx.x + 1) / gridDim.x);
    for (int i = i0; i < i1;) {
        const int q = map.seq_of(i), first = map.first_of(q);
        const Span sp = map.span_at(q);
        const int end = first + static_cast<int>(chunks_of(sp)), next = end < i1 ? end : i1;
        const int pair = a.halves ? q % a.n_pairs : q / 2;
        const int side = a.halves ? q / a.n_pairs : q % 2;
        const bool write = side == 0 && i == first;
        if (write || (a.grad && pair != have)) {
            slopes_of(pair, write);
            have = pair;
        }
        const int64_t b = sp.b + static_cast<int64_t>(i - first) * kChunk;
        int64_t e = sp.b + static_cast<int64_t>(next - first) * kChunk;
        if (e > sp.e) e = sp.e;
        i = next;
        if (!a.grad) continue;
        const float g = slope[side];
#pragma unroll 4
        for (int64_t t = b + threadIdx.x; t < e; t += kThreads)
            a.grad[t] = (a.active && a.active[t] == 0) ? 0.0f : g;
    }
    if (a.grad) {
        // tokens before the first and behind the last sequence
        const int64_t who = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
        const int64_t all = static_cast<int64_t>(gridDim.x) * kThreads;
        const int64_t head = map.span_at(0).b, tail = map.span_at(2 * a.n_pairs - 1).e;
        for (int64_t t = who; t < head; t += all) a.grad[t] = 0.0f;
        for (int64_t t = tail + who; t < a.T; t += all) a.grad[t] = 0.0f;
    }
    // the last CTA to come here adds up the pairs, whose losses the CTAs' first threads have written
    if (threadIdx.x == 0) {
        __threadfence();
        last_here = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    }
    __syncthreads();
    if (!last_here) return;
    __threadfence();
    preference_finish(a, a.out_pair_loss, map.bad, scratch.tmp[0]);
}

cudaError_t launch_clusters(const PreferenceCall& a, int clusters, int size, int team, int alone, int threads,
                            cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * size), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, k_preference, a, team, alone);
}

cudaError_t launch_after(void (*kernel)(PreferenceCall), int blocks, const PreferenceCall& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

bool preference_split(int64_t T, int64_t n_pairs) {
    return n_pairs > 0 && 2 * n_pairs <= kSplitSeqs && T / n_pairs >= kPreferenceSplitTokens;
}

int64_t preference_chunks(int64_t T, int64_t n_pairs) { return T / kChunk + 2 * n_pairs; }

cudaError_t launch_preference_loss(const PreferenceArgs& args, int num_sms, cudaStream_t stream) {
    PreferenceCall a;
    static_cast<PreferenceArgs&>(a) = args;
    a.smooth32 = static_cast<float>(a.label_smoothing);
    a.keep32 = static_cast<float>(1.0 - a.label_smoothing);
    a.beta2 = split_two(a.beta);
    a.margin2 = split_two(a.margin);
    // 1 / (2 beta) beyond fp32 is its largest number: it must not meet an infinite h as infinity
    a.half_over_beta2 = split_two(fmin(a.half_over_beta, double(std::numeric_limits<float>::max())));
    a.scale2 = split_two(a.scale_per_pair);
    if (a.n_pairs == 0) {
        if (a.grad && a.T > 0) {
            const cudaError_t e = cudaMemsetAsync(a.grad, 0, size_t(a.T) * sizeof(float), stream);
            if (e != cudaSuccess) return e;
        }
        return launch_clusters(a, 1, 1, 1, 1, 128, stream);
    }
    const int64_t mean = a.T / a.n_pairs;  // tokens of a pair, about
    // 128 threads against 512: 5.3 and 5.6 us at 512 tokens a pair, 6.4 and 5.9 at 1024, 8.9 and 6.5 at
    // 2048 (4 pairs); 8.8 and 13.3, 10.6 and 14.2, 14.7 and 16.0 (512 pairs)
    const int threads = mean <= 1024 ? 128 : kThreads;
    if (a.T <= kPreferenceClusterTokens && a.n_pairs <= kCluster) {
        // a CTA for every pair, and several where the pairs are long and few: with 2048, 4096 and 8192
        // tokens a CTA 7.9, 7.6 and 7.5 us for one pair of 4096, 10.1, 10.0 and 10.4 for four of 8192
        int size = 1, team = 1;
        while (size < kCluster && size < a.n_pairs) size *= 2;
        while (size < kCluster && mean / team > kThreads * 8) {
            size *= 2;
            team *= 2;
        }
        return launch_clusters(a, 1, size, team, 1, threads, stream);
    }
    if (preference_split(a.T, a.n_pairs)) {
        const int64_t chunks = preference_chunks(a.T, a.n_pairs);
        const int64_t need = (chunks + kWarps - 1) / kWarps;
        const int most = num_sms * 3;
        k_preference_chunks<<<static_cast<int>(need < most ? need : most), kThreads, 0, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return launch_after(k_preference_spread, static_cast<int>(need < num_sms * 2 ? need : num_sms * 2), a, stream);
    }
    // CTAs per pair: enough to fill the device, and none with less than 4096 tokens.  With 2048, 4096
    // and 8192: 8.8, 8.4 and 8.4 us for 16 pairs of 4096 tokens, 8.6, 10.7 and 10.6 of 8192, 10.0, 10.8
    // and 14.0 of 16384; 19.6, 14.4 and 15.9 for 64 of 16384; 11.4, 9.3 and 9.3 for 152 of 4096
    int team = 1;
    while (team < kCluster && static_cast<int64_t>(a.n_pairs) * team < num_sms * 2 && mean / (2 * team) >= 4096) team *= 2;
    const int64_t most = static_cast<int64_t>(num_sms) * 64 / team;
    const cudaError_t e = launch_clusters(a, static_cast<int>(a.n_pairs < most ? a.n_pairs : most), team, team, 0,
                                          threads, stream);
    if (e != cudaSuccess) return e;
    return launch_after(k_preference_final, 1, a, stream);
}

}  // namespace rlk
