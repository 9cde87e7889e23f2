// Verification of drafted tokens against the target's probabilities.
//
// The rows' tile pairs come from the materialised-logits pass.  One cluster per
// sequence does the rest in one launch:
//
//   rows    a CTA merges its rows' tile pairs along the contract's tree, and
//           decides a drafted token where the row has one: accepted where
//           u q(x) < p(x);
//   draw    the row of the first refusal, or the row behind the last draft, is
//           split over the CTAs: argmax_v w(v) / e(v) with w = max(p - q, 0), or p.
//
// A draw by a race of exponentials is a maximum, so its result does not depend
// on how the vocabulary is split over threads and CTAs; the lowest token wins a
// tie.  p = e^(l - m) / s and q = e^(d - draft_lse) are formed from exact
// differences (a rounded value and its error), since l - m alone, rounded,
// would cost 2^-21 of p at l - m = -16.
//
// The draw goes over a row once with an upper bound of each token's w / e, from
// the hardware's approximate exponentials and reciprocal (2^-15 off at most, with
// 2^-13 of p and of q to spare), and each thread keeps its two largest.  The
// first ones alone are formed exactly, side by side, and then the second ones that
// reach the best weight found; a thread that has had a third one which does goes
// over its tokens again, which is seldom.
//
// What bounds it: for large batches HBM first and the draw's instructions next
// (256 sequences of up to 8 drafts, V = 151936, fp32: 230 us with the row sums, 137 of
// them theirs, 0.70 of the copy rate on the bytes of both); for small ones latency:
// one sequence of 4 bf16 drafts 17 us, 5 of them the row sums', 64 sequences of
// up to 7 looked-up drafts at V = 50257 37.5, 23 of them the row sums'; 8 and 32 sequences of up to 8 at V =
// 151936 21 and 38 in bf16, 30 and 50 in fp32; 256 in bf16 167 (floor 92), with the draft's log-probabilities in
// fp32 172 (102).  Splitting a
// sequence over a cluster and not over the grid keeps the draw's meeting in distributed
// shared memory, in the same launch.
#include <cooperative_groups.h>
#include <cstdint>
#include <type_traits>

#include "rlk_block.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"
#include "rlk_tree.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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

// A row's pair and log-sum-exp.
struct RowSum {
    float m, s, lse;
};

// What is drawn from: a target row, a draft row or a certain token to take off, the noise.
struct Draw {
    const uint8_t* target;  // first logit of the row
    const uint8_t* draft;   // of the draft's row, or nullptr
    const float* noise;
    float m, s, draft_lse;
    int certain;            // token with q = 1, or -1
    bool from_target;       // p exceeds q nowhere: drawn from p, where q is a number

    // the draft's row as far as the bounds go
    __device__ __forceinline__ const uint8_t* taken_off() const { return from_target ? nullptr : draft; }
};

// The weight of a token, exactly as defined, over its noise; 0 where there is none.
__device__ __noinline__ float weight_of(const VerifyArgs& a, const Draw& r, int v) {
    const float l = logit_at(r.target, a.target_dtype, v), e = r.noise[v];
    float w = __fdiv_rn(exp_diff(l, r.m), r.s);
    if (r.draft) {
        const float q = exp_diff(logit_at(r.draft, a.draft_dtype, v), r.draft_lse);
        if (!r.from_target || q != q) w = __fsub_rn(w, q);  // NaN is no weight
    } else if (v == r.certain) {
        w = __fsub_rn(w, 1.0f);
    }
    return w > 0.0f ? __fdiv_rn(w, e) : 0.0f;
}

__device__ __forceinline__ uint32_t bytes_of(int dtype) { return dtype == RLK_DTYPE_F32 ? 4 : 2; }

// A chunk of kChunk tokens: a thread's are 4 consecutive ones of each half of it where it is read in
// 16-byte (bf16: 8-byte) vectors, else every 256th.
constexpr int kChunk = kThreads * kAhead;
template <bool kVec>
__device__ __forceinline__ int token_at(int base, int k) {
    return kVec ? base + (k >> 2) * (4 * kThreads) + static_cast<int>(threadIdx.x) * 4 + (k & 3)
                : base + k * kThreads + static_cast<int>(threadIdx.x);
}

// The bounds' constants: base-2 logarithms of 1 + 2^-13 and of 1 - 2^-13, and of e.
constexpr float kLog2e = 0x1.715476p+0f, kMore = 0x1.715p-13f, kLess = -0x1.716p-13f;
struct Scale {
    float m, log_more, draft_lse;
};
// At least w / e, NaN where the noise or the draft's logit is not a number (or p was flushed to 0 and e's
// reciprocal is infinite).
template <bool kDraft>
__device__ __forceinline__ float bound_of(float l, float e, float d, const Scale& c) {
    float p = approx_exp2(__fmaf_rn(__fsub_rn(l, c.m), kLog2e, c.log_more));
    if (kDraft) p = __fsub_rn(p, approx_exp2(__fmaf_rn(__fsub_rn(d, c.draft_lse), kLog2e, kLess)));
    return __fmul_rn(p, approx_rcp(e));
}
__device__ __forceinline__ float min_or_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// Whether a factor of the bound may have been flushed to 0, so that it says nothing.  (p and q that cancel
// give a bound of 0 too, which is one.)  Below -105 p itself is 0, and infinite noise leaves no weight.
__device__ __forceinline__ bool unsure(float l, float e, const Scale& c) {
    const float d = __fsub_rn(l, c.m);
    return d >= -105.0f && (approx_exp2(__fmaf_rn(d, kLog2e, c.log_more)) < 0x1p-100f || (e >= 0x1p100f && e < CUDART_INF_F));
}

// The three largest bounds of a thread's tokens, and whose the first two are.  (With one token kept, a
// likely token that the draft finds a little likelier still would often hide a better one.)
struct Seen {
    float top = -1.0f, second = -1.0f, third = -1.0f;
    int at = -1, second_at = -1;
    __device__ __forceinline__ void see(float bound, int v) {
        const bool first = bound > top, ahead = bound > second;
        third = fmaxf(third, fminf(bound, second));
        second_at = first ? at : ahead ? v : second_at;
        second = fmaxf(second, fminf(bound, top));
        at = first ? v : at;
        top = fmaxf(top, bound);
    }
};
// Tokens k0, k0 + 1, .. of a thread's part of a chunk.
template <bool kVec, bool kDraft, int kN>
__device__ __forceinline__ void see_tokens(const Scale& c, int base, int k0, int v1, const float (&l)[kN], const float (&e)[kN],
                                           const float (&d)[kN], Seen& seen) {
    float bound[kN], least = CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        bound[k] = bound_of<kDraft>(l[k], e[k], d[k], c);
        least = min_or_nan(least, fabsf(bound[k]));
        bound[k] = fmaxf(bound[k], -1.0f);  // no token: of NaN and -1 the latter
        if (!kVec && token_at<kVec>(base, k0 + k) >= v1) bound[k] = -1.0f;
    }
    if (!(least >= 0x1p-100f)) {
#pragma unroll
        for (int k = 0; k < kN; ++k)
            if ((kVec || token_at<kVec>(base, k0 + k) < v1) && unsure(l[k], e[k], c)) seen.third = CUDART_INF_F;
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) seen.see(bound[k], token_at<kVec>(base, k0 + k));
}

// 4 consecutive values of a row, as they lie in memory.
template <int kDtype>
struct Four {
    using Words = typename std::conditional<kDtype == RLK_DTYPE_F32, float4, uint2>::type;
    Words w;
    __device__ __forceinline__ void load(const uint8_t* row, int v) {
        w = *reinterpret_cast<const Words*>(row + static_cast<int64_t>(v) * (sizeof(Words) / 4));
    }
    __device__ __forceinline__ void values(float (&x)[4]) const {
        if constexpr (kDtype == RLK_DTYPE_F32) {
            x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
        } else {
            x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
        }
    }
};
constexpr int kNoDraft = -1;

// Looks over whole chunks [v0, v1) whose rows start at 16 bytes; the next chunk is on its way while one
// is worked on.
template <int kTarget, int kDraft>
__device__ __forceinline__ Seen look_vec(const uint8_t* target, const uint8_t* noise, const uint8_t* draft, float m, float log_more,
                                      float draft_lse, int v0, int v1) {
    const Scale c = {m, log_more, draft_lse};
    constexpr int kD = kDraft == kNoDraft ? RLK_DTYPE_BF16 : kDraft;
    Seen seen;
    Four<kTarget> t[2];
    Four<RLK_DTYPE_F32> n[2];
    Four<kD> q[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int v = token_at<true>(v0, 4 * g);
        t[g].load(target, v);
        n[g].load(noise, v);
        if (kDraft != kNoDraft) q[g].load(draft, v);
    }
#pragma unroll 1
    for (int base = v0; base < v1; base += kChunk) {
        const int next = base + kChunk < v1 ? base + kChunk : base;  // the last chunk once more
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float l[4], e[4], d[4];
            t[g].values(l);
            n[g].values(e);
            if (kDraft != kNoDraft) q[g].values(d);
            const int v = token_at<true>(next, 4 * g);
            t[g].load(target, v);
            n[g].load(noise, v);
            if (kDraft != kNoDraft) q[g].load(draft, v);
            see_tokens<true, kDraft != kNoDraft>(c, base, 4 * g, v1, l, e, d, seen);
        }
    }
    return seen;
}
// Looks any tokens [v0, v1) over.
__device__ __noinline__ Seen look_plain(const VerifyArgs& a, const Draw& r, float log_more, int v0, int v1, Seen seen) {
    const Scale c = {r.m, log_more, r.draft_lse};
    const uint8_t *const target = r.target, *const draft = r.taken_off();
    const float* const noise = r.noise;
#pragma unroll 1
    for (int base = v0; base < v1; base += kChunk) {
        float l[kAhead], e[kAhead], d[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int v = min(token_at<false>(base, k), v1 - 1);
            l[k] = logit_at(target, a.target_dtype, v);
            e[k] = noise[v];
            d[k] = draft ? logit_at(draft, a.draft_dtype, v) : 0.0f;
        }
        if (draft) see_tokens<false, true>(c, base, 0, v1, l, e, d, seen);
        else see_tokens<false, false>(c, base, 0, v1, l, e, d, seen);
    }
    return seen;
}
// A thread's tokens again, each whose weight may reach `known` formed exactly.
template <bool kVec>
__device__ __noinline__ uint64_t look_again(const VerifyArgs& a, const Draw& r, float log_more, int v0, int v1, float known) {
    const Scale c = {r.m, log_more, r.draft_lse};
    uint64_t best = 0;
#pragma unroll 1
    for (int base = v0; base < v1; base += kChunk) {
        uint32_t may = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int v = token_at<kVec>(base, k), at = min(v, v1 - 1);
            const float l = logit_at(r.target, a.target_dtype, at), e = r.noise[at];
            const float b = r.taken_off() ? bound_of<true>(l, e, logit_at(r.draft, a.draft_dtype, at), c)
                                          : bound_of<false>(l, e, 0.0f, c);
            may |= v < v1 && ((b >= 0.0f && b >= known) || unsure(l, e, c)) ? 1u << k : 0u;
        }
        for (; may; may &= may - 1) {
            const int v = token_at<kVec>(base, __ffs(may) - 1);
            const float w = weight_of(a, r, v);
            if (w > 0.0f) best = max_key(best, key_of(w, v));
        }
    }
    return best;
}

// The cluster's finds: the first refused row of each CTA (n where there is none) with its sums, and
// those of the row behind the last draft.
struct Found {
    int first;
    RowSum sum, last;
};

// Four CTAs an SM leave 64 registers: with target and draft in fp32 (and without a draft, whose type is taken as
// fp32) 24 to 32 bytes a thread are spilled, with one of them in fp32 8 to 16.
template <int kLogL, int kTarget, int kDraft>
__global__ void __launch_bounds__(kThreads, 4) k_draft_verify(const __grid_constant__ VerifyArgs a) {
    __shared__ MaxSum node[kWarps][kWarps];  // [row][warp]
    __shared__ bool node_held[kWarps][kWarps];
    __shared__ RowSum row_sum[kWarps];
    __shared__ bool row_ok[kWarps];
    __shared__ uint64_t warp_best[kWarps];
    __shared__ uint64_t cta_best;
    __shared__ Found found;
    __shared__ uint32_t best_w;  // the best weight formed so far, as its bits
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int s = static_cast<int>(blockIdx.x) / ctas, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int o0 = a.offsets[s], o1 = a.offsets[s + 1];
    if (o0 < 0 || o1 < o0 || o1 > a.n_draft) {
        ptx::grid_dependency_wait();  // what the call before this one may still be reading is not written earlier
        if (rank == 0 && threadIdx.x == 0) {
            a.out_accepted[s] = -1;
            report_status(a.status, RLK_ERR_INVALID_ARG);
        }
        return;
    }
    const int n = o1 - o0;
    const int64_t row0 = static_cast<int64_t>(o0) + s;
    if (a.active && a.active[s] == 0) {
        ptx::grid_dependency_wait();
        if (rank != 0) return;
        if (threadIdx.x == 0) a.out_accepted[s] = 0;
        for (int i = threadIdx.x; i <= n; i += kThreads) {
            a.out_tokens[row0 + i] = -1;
            a.out_logprob[row0 + i] = 0.0f;
        }
        return;
    }
    if (threadIdx.x == 0) found.first = n;
    // the drafted token of the row that this warp finishes, its logits and number, in lane 0: on their way while
    // the trees are merged
    int x;
    float l, q, u;
    auto read_draft = [&](int own) {
        x = -1;
        l = u = 0.0f;
        q = 1.0f;
        if (lane == 0 && own < n) {
            x = a.tokens[o0 + own];
            u = a.uniforms[o0 + own];
            if (x < 0 || x >= a.V) x = -1;
            if (x >= 0) {
                l = logit_at(a.target, a.target_dtype, (row0 + own) * a.ld_target + x);
                if (a.draft)
                    q = exp_diff(logit_at(a.draft, a.draft_dtype, (static_cast<int64_t>(o0) + own) * a.ld_draft + x),
                                 a.draft_lse ? a.draft_lse[o0 + own] : 0.0f);
            }
        }
    };
    read_draft(rank + warp * ctas);
    const int per = ((a.V + ctas - 1) / ctas + 7) / 8 * 8;
    const int v0 = min(a.V, rank * per), v1 = min(a.V, v0 + per);
    if (a.fetch_noise) {  // this CTA's part of the row, while the trees are merged
        const float* const noise = a.noise + s * a.ld_noise;
        for (int v = v0 + 32 * static_cast<int>(threadIdx.x); v < v1; v += 32 * kThreads)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + v) : "memory");
    }
    const SlotRun run = slot_run<8>(threadIdx.x, a.depth, a.n_tiles);
    ptx::grid_dependency_wait();  // the tile pairs are the previous kernel's output
    // this CTA's rows, every ctas-th one, up to 8 at a time: all threads merge each row's pairs as far as
    // their warps go, then a warp a row finishes it and decides
    for (int i0 = rank; i0 <= n; i0 += ctas * kWarps) {
        const int own = i0 + warp * ctas;  // the row that this warp finishes
        if (i0 != rank) read_draft(own);
        for (int j = 0; j < kWarps && i0 + j * ctas <= n; ++j) {
            const float2* row = a.partials + (row0 + i0 + j * ctas) * a.n_tiles;
            bool held;
            MaxSum v = merge_run<kLogL>(run, [&](int k) { return row[k]; }, held);
#pragma unroll 1
            for (int lv = 0; lv < 5; ++lv) v = shuffle_level(v, held, lane, lv);
            if (lane == 0) {
                node[j][warp] = v;
                node_held[j][warp] = held;
            }
        }
        __syncthreads();
        if (own <= n) {
            MaxSum v = node[warp][lane & (kWarps - 1)];
            bool held = node_held[warp][lane & (kWarps - 1)];
#pragma unroll 1
            for (int lv = 0; lv < 3; ++lv) v = shuffle_level(v, held, lane, lv);
            if (lane == 0) {
                const RowSum sum = {v.m, v.s, __fadd_rn(v.m, contract_log(v.s))};
                const bool ok = x >= 0 && __fmul_rn(u, q) < __fdiv_rn(exp_diff(l, v.m), v.s);
                row_sum[warp] = sum;
                row_ok[warp] = ok;
                if (ok) {  // rows behind a refusal are set right at the end
                    a.out_tokens[row0 + own] = x;
                    a.out_logprob[row0 + own] = __fsub_rn(l, sum.lse);
                }
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int j = 0; j < kWarps && i0 + j * ctas <= n && found.first == n; ++j) {
                const int i = i0 + j * ctas;
                if (i == n) {
                    found.last = row_sum[j];
                } else if (!row_ok[j]) {
                    found.first = i;
                    found.sum = row_sum[j];
                }
            }
        }
        __syncthreads();
        if (found.first < n) break;  // what is behind it is not looked at
    }
    cluster.sync();
    // a lane per CTA
    const Found* const other = cluster.map_shared_rank(&found, lane < ctas ? lane : 0);
    const int acc = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<uint32_t>(other->first)));
    const RowSum& theirs = acc < n ? other->sum : other->last;
    const int owner = acc % ctas;  // rows go to the CTAs in turn
    RowSum sum;
    sum.m = __shfl_sync(0xffffffffu, theirs.m, owner);
    sum.s = __shfl_sync(0xffffffffu, theirs.s, owner);
    sum.lse = __shfl_sync(0xffffffffu, theirs.lse, owner);
    const int refused = acc < n ? a.tokens[o0 + acc] : -1;
    // in shared memory for what is seldom called and reads it there, in registers for the rest
    __shared__ Draw shared_draw;
    Draw r;
    r.target = static_cast<const uint8_t*>(a.target) + (row0 + acc) * a.ld_target * bytes_of(a.target_dtype);
    r.noise = a.noise + s * a.ld_noise;
    r.m = sum.m;
    r.s = sum.s;
    r.draft = acc < n && a.draft
                  ? static_cast<const uint8_t*>(a.draft) + (static_cast<int64_t>(o0) + acc) * a.ld_draft * bytes_of(a.draft_dtype)
                  : nullptr;
    r.draft_lse = r.draft && a.draft_lse ? a.draft_lse[o0 + acc] : 0.0f;
    r.certain = a.draft ? -1 : refused;
    r.from_target = false;
    const bool vec = ((reinterpret_cast<uintptr_t>(r.target) | reinterpret_cast<uintptr_t>(r.noise) |
                       reinterpret_cast<uintptr_t>(r.draft)) & 15) == 0;
    // not a distribution: a NaN or +infinity in the row, or nothing but -infinity
    const bool usable = fabsf(r.m) < CUDART_INF_F && r.s > 0.0f && r.s < CUDART_INF_F;
    // what is read in vectors: whole chunks
    const int by_vec = vec ? v0 + (v1 - v0) / kChunk * kChunk : v0;
    const float log_more = __fmaf_rn(-kLog2e, usable ? contract_log(r.s) : 0.0f, kMore);
    uint64_t best = 0;
    // a second time from p where p exceeds q nowhere
    for (int pass = 0; usable && pass < 2 && best == 0; ++pass) {
        if (pass == 1) {
            if (acc == n) break;
            r.from_target = true;
            r.certain = -1;
            cluster.sync();  // everyone has read the first pass's keys
        }
        if (threadIdx.x == 0) {
            best_w = 0;
            shared_draw = r;
        }
        __syncthreads();
        Seen seen;
        if (by_vec > v0) {
            const uint8_t* const noise = reinterpret_cast<const uint8_t*>(r.noise);
            seen = r.taken_off() ? look_vec<kTarget, kDraft>(r.target, noise, r.draft, r.m, log_more, r.draft_lse, v0, by_vec)
                                 : look_vec<kTarget, kNoDraft>(r.target, noise, nullptr, r.m, log_more, 0.0f, v0, by_vec);
        }
        if (by_vec < v1) seen = look_plain(a, shared_draw, log_more, by_vec, v1, seen);
        uint64_t mine = 0;
        if (seen.top >= 0.0f) {
            const float w = weight_of(a, shared_draw, seen.at);
            if (w > 0.0f) mine = key_of(w, seen.at);
        }
        const uint32_t warp_w = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32));
        __syncthreads();
        if (lane == 0 && warp_w) atomicMax(&best_w, warp_w);
        __syncthreads();
        const float known = __uint_as_float(best_w);
        if (seen.second >= 0.0f && seen.second >= known) {
            const float w = weight_of(a, shared_draw, seen.second_at);
            if (w > 0.0f) mine = max_key(mine, key_of(w, seen.second_at));
        }
        if (seen.third >= 0.0f && seen.third >= known) {
            if (by_vec > v0) mine = max_key(mine, look_again<true>(a, shared_draw, log_more, v0, by_vec, known));
            if (by_vec < v1) mine = max_key(mine, look_again<false>(a, shared_draw, log_more, by_vec, v1, known));
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mine = max_key(mine, __shfl_xor_sync(0xffffffffu, mine, o));
        if (lane == 0) warp_best[warp] = mine;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mine = max_key(mine, warp_best[w]);
            cta_best = mine;
        }
        cluster.sync();
        best = *cluster.map_shared_rank(&cta_best, lane < ctas ? lane : 0);
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
        best = __shfl_sync(0xffffffffu, best, 0);
    }
    if (rank == 0) {
        const int drawn = best != 0 ? static_cast<int>(~static_cast<uint32_t>(best)) : -1;
        for (int i = acc + threadIdx.x; i <= n; i += kThreads) {
            a.out_tokens[row0 + i] = i == acc ? drawn : -1;
            float lp = 0.0f;
            if (i == acc) lp = drawn >= 0 ? __fsub_rn(logit_at(r.target, a.target_dtype, drawn), sum.lse) : CUDART_NAN_F;
            a.out_logprob[row0 + i] = lp;
        }
        if (threadIdx.x == 0) {
            a.out_accepted[s] = acc;
            if (drawn < 0) report_status(a.status, RLK_ERR_NONFINITE);
            if (acc < n && (refused < 0 || refused >= a.V)) report_status(a.status, RLK_ERR_TARGET_RANGE);
        }
    }
    cluster.sync();  // nobody leaves while its shared memory may be read
}

template <int kLogL, int kTarget, int kDraft>
cudaError_t launch(const VerifyArgs& a, int ctas, cudaStream_t stream) {
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
    return cudaLaunchKernelEx(&cfg, k_draft_verify<kLogL, kTarget, kDraft>, a);
}

template <int kTarget, int kDraft>
cudaError_t launch_types(const VerifyArgs& a, int ctas, cudaStream_t stream) {
    switch (a.depth > 8 ? a.depth - 8 : 0) {
        case 0: return launch<0, kTarget, kDraft>(a, ctas, stream);
        case 1: return launch<1, kTarget, kDraft>(a, ctas, stream);
        case 2: return launch<2, kTarget, kDraft>(a, ctas, stream);
        case 3: return launch<3, kTarget, kDraft>(a, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_draft_verify(const VerifyArgs& args, int num_sms, cudaStream_t stream) {
    VerifyArgs a = args;
    // the noise is fetched ahead where all of it is half of the second-level cache at most (64 MB): 64 sequences
    // at V = 50257 37.3 instead of 38.3 us, 16 at V = 151936 36.6 instead of 37.4
    a.fetch_noise = static_cast<int64_t>(a.n_seqs) * a.V <= (int64_t(1) << 24);
    // up to 8 CTAs a sequence, as long as all of them are resident at once (4 per SM).  Against 4 and 16
    // of them, side by side: one sequence at V = 151936 16.8 us (22.0, 15.8), at V = 1000 11.7 (12.3, 12.9), 16
    // at V = 32000 17.0 (18.3, 20.7), 32 at V = 2000 14.0 (13.7, 21.1).
    int ctas = 8;
    while (ctas > 1 && static_cast<int64_t>(a.n_seqs) * ctas > 4 * static_cast<int64_t>(num_sms)) ctas /= 2;
    const bool draft_f32 = a.draft_dtype == RLK_DTYPE_F32;
    if (a.target_dtype == RLK_DTYPE_F32)
        return draft_f32 ? launch_types<RLK_DTYPE_F32, RLK_DTYPE_F32>(a, ctas, stream)
                         : launch_types<RLK_DTYPE_F32, RLK_DTYPE_BF16>(a, ctas, stream);
    return draft_f32 ? launch_types<RLK_DTYPE_BF16, RLK_DTYPE_F32>(a, ctas, stream)
                     : launch_types<RLK_DTYPE_BF16, RLK_DTYPE_BF16>(a, ctas, stream);
}

}  // namespace rlk
