// Backward of the block norms.  Per row, with dy = grad_out, x the residual
// stream that was normed, b the block's output, z its gate,
//
//   up_i = dy_i gamma_pre_i        c = rstd_x^2 / H sum_i up_i x_i
//   dx_i = rstd_x (up_i - x_i c) + grad_residual_out_i
//   grad_residual_i = rs dx_i      d_i = bs dx_i
//   n_i  = b_i rstd_b gamma_post_i           grad_gate_i = d_i n_i gate'(z_i)
//   v_i  = d_i gate(z_i) gamma_post_i        k = rstd_b^2 / H sum_i v_i b_i
//   grad_block_i = rstd_b (v_i - b_i k)
//   grad_gamma_pre_i  = sum over rows of dy_i x_i rstd_x
//   grad_gamma_post_i = sum over rows of d_i gate(z_i) b_i rstd_b
//
// The sums over a row are the forward's trees (the squares) or chains of 16
// features and a tree (the products).  A row's gradients do not depend on the
// batch around it.  The grad_gammas are summed over at most 152 ranges of
// consecutive rows, one CTA each, in chains of 64 rows a team, then over the
// ranges by a second launch, in an order that T and H fix.
//
// Element i = 512 w + 256 g + 8 l + j is warp w's lane l's j-th value of its
// column group g, as in the forward.
//
// What bounds it: HBM.
#pragma once

#include <atomic>
#include <cstdint>

#include "rlk_block.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 512;  // of a CTA, one CTA per SM
constexpr int kStages = 2;     // a row flies while another is worked on
constexpr int kChain = 64;     // rows that a team adds one after the other before it starts a new sum
constexpr size_t kHeldBytes = size_t(kThreads) * 32 * sizeof(float);

// 16-byte places of a thread's ring in one stage: 16 features of each tensor.
template <int kGo, int kSaved>
struct Ring {
    static constexpr int kGoPlaces = kGo == RLK_DTYPE_F32 ? 4 : 2;
    static constexpr int kSavedPlaces = kSaved == RLK_SAVED_BF16 ? 2 : 1;
    static constexpr int kX = kGoPlaces, kBlock = kX + kSavedPlaces, kGate = kBlock + kSavedPlaces;
    static constexpr int kRes = kGate + kSavedPlaces;
    // where all of them do not fit into 227 KB the residual's gradient is read as it is needed
    static constexpr bool kHasRes = !(kGo == RLK_DTYPE_F32 && kSaved == RLK_SAVED_BF16);
    static constexpr int kPlaces = kRes + (kHasRes ? 2 : 0);
    static constexpr size_t kBytes = size_t(kStages) * kPlaces * kThreads * sizeof(uint4);
    static_assert(kBytes + kHeldBytes + 1024 <= 232448, "the ring and the sums fit into shared memory");
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void pairs_of(uint4 w, uint64_t (&v)[4]) {
    v[0] = unpack_bf16x2(w.x);
    v[1] = unpack_bf16x2(w.y);
    v[2] = unpack_bf16x2(w.z);
    v[3] = unpack_bf16x2(w.w);
}
__device__ __forceinline__ uint64_t pair_of_words(uint32_t lo, uint32_t hi) {
    return f2_pack(__uint_as_float(lo), __uint_as_float(hi));
}

// 8 features of a gradient at element i.
__device__ __forceinline__ void load_grad(const void* base, int dtype, int64_t i, uint64_t (&v)[4]) {
    if (dtype == RLK_DTYPE_F32) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
        const uint4 a = p[0], b = p[1];
        v[0] = pair_of_words(a.x, a.y);
        v[1] = pair_of_words(a.z, a.w);
        v[2] = pair_of_words(b.x, b.y);
        v[3] = pair_of_words(b.z, b.w);
    } else {
        pairs_of(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i), v);
    }
}
__device__ __forceinline__ void store_grad(void* base, int dtype, int64_t i, const uint64_t (&v)[4]) {
    if (dtype == RLK_DTYPE_F32) {
        float e[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) f2_unpack(v[p], e[2 * p], e[2 * p + 1]);
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(e[0], e[1], e[2], e[3]);
        p[1] = make_float4(e[4], e[5], e[6], e[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
            make_uint4(pack_bf16x2(v[0]), pack_bf16x2(v[1]), pack_bf16x2(v[2]), pack_bf16x2(v[3]));
    }
}

// gate(z) and gate'(z) for a pair.  With e = e^-|z|, which does not overflow, the sigmoid is 1 or
// e over 1 + e and its slope e over (1 + e)^2.
__device__ __forceinline__ void gate_of(int kind, uint64_t z, uint64_t& gate, uint64_t& slope) {
    if (kind != RLK_GATE_SIGMOID) {
        gate = z;
        slope = f2_splat(1.0f);
        return;
    }
    float v[2], g[2], s[2];
    f2_unpack(z, v[0], v[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float e = exp_any(-fabsf(v[k])), r = __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
        g[k] = v[k] < 0.0f ? __fmul_rn(e, r) : r;
        s[k] = __fmul_rn(__fmul_rn(e, r), r);
    }
    gate = f2_pack(g[0], g[1]);
    slope = f2_pack(s[0], s[1]);
}

// A team of kWarps warps (a power of two) takes a row, a CTA's teams every kTeams-th row of its
// range.  A thread copies its own features of the next row into its own places of a ring of shared
// memory, which needs no barrier; the copies fly while the current row is reduced.
template <int kWarps, int kGo, int kSaved>
__global__ void __launch_bounds__(kThreads, 1) k_block_norm_backward(const BlockBwdArgs a) {
    using R = Ring<kGo, kSaved>;
    constexpr int kTeams = kThreads / 32 / kWarps;
    static_assert(kWarps == 1 || kTeams <= 15, "a named barrier (1 .. 15) per team");
    extern __shared__ uint4 ring[];  // [stage][place][thread]
    __shared__ __align__(16) float4 part[2][kThreads / 32];
    ptx::grid_dependents_launch();
    const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * kWarps);
    const int warp = (threadIdx.x >> 5) % kWarps;
    const int i0 = 512 * warp + 8 * lane;  // and i0 + 256
    const bool in[2] = {i0 < a.H, i0 + 256 < a.H};
    const int64_t r0 = static_cast<int64_t>(a.T) * blockIdx.x / gridDim.x;
    const int64_t r1 = static_cast<int64_t>(a.T) * (blockIdx.x + 1) / gridDim.x;
    const bool pow2 = (a.H & (a.H - 1)) == 0;
    const float h = static_cast<float>(a.H), inv_h = __fdiv_rn(1.0f, h);
    const int odd = lane & 1;
    const bool branch = a.block.data != nullptr, post = a.gamma_post != nullptr, gated = a.gate.data != nullptr;
    const bool res_in_ring = R::kHasRes && a.grad_res && a.gx_dtype == RLK_DTYPE_BF16;
    auto place = [&](int stage, int k) { return ring + (stage * R::kPlaces + k) * kThreads + threadIdx.x; };

    auto fetch_saved = [&](const SavedIn& s, int64_t i, int stage, int k, int g) {
        if (kSaved == RLK_SAVED_BF16)
            copy16(place(stage, k + g), static_cast<const uint16_t*>(s.data) + i);
        else
            copy8(reinterpret_cast<uint2*>(place(stage, k)) + g, static_cast<const uint8_t*>(s.data) + i);
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < r1) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!in[g]) continue;
                const int64_t i = t * a.H + i0 + 256 * g;
                if (kGo == RLK_DTYPE_F32) {
                    copy16(place(stage, 2 * g), static_cast<const float*>(a.grad_out) + i);
                    copy16(place(stage, 2 * g + 1), static_cast<const float*>(a.grad_out) + i + 4);
                } else {
                    copy16(place(stage, g), static_cast<const uint16_t*>(a.grad_out) + i);
                }
                fetch_saved(a.x, i, stage, R::kX, g);
                if (branch) fetch_saved(a.block, i, stage, R::kBlock, g);
                if (gated) fetch_saved(a.gate, i, stage, R::kGate, g);
                if (res_in_ring) copy16(place(stage, R::kRes + g), static_cast<const uint16_t*>(a.grad_res) + i);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the bytes of this thread's blocks of 32 features, a row ahead
    uint32_t next[3][2] = {};
    auto fetch_scales = [&](int64_t t) {
        if constexpr (kSaved != RLK_SAVED_BF16) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!in[g] || t >= r1) continue;
                const int64_t k = (t * a.H + i0 + 256 * g) >> 5;
                next[0][g] = a.x.scales[k];
                if (branch) next[1][g] = a.block.scales[k];
                if (gated) next[2][g] = a.gate.scales[k];
            }
        }
    };
    uint4 gam_pre[2] = {}, gam_post[2] = {};
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (in[g]) gam_pre[g] = *reinterpret_cast<const uint4*>(a.gamma_pre + i0 + 256 * g);
        if (in[g] && post) gam_post[g] = *reinterpret_cast<const uint4*>(a.gamma_post + i0 + 256 * g);
    }
    uint64_t d_pre[2][4] = {}, d_post[2][4] = {};
    ulonglong2* const held = reinterpret_cast<ulonglong2*>(ring + kStages * R::kPlaces * kThreads) + threadIdx.x;
    auto each_held = [&](auto fn) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            fn(held[k * kThreads], d_pre[k >> 1][2 * (k & 1)], d_pre[k >> 1][2 * (k & 1) + 1]);
            fn(held[(4 + k) * kThreads], d_post[k >> 1][2 * (k & 1)], d_post[k >> 1][2 * (k & 1) + 1]);
        }
    };
    auto add_held = [&] {
        each_held([](const ulonglong2& v, uint64_t& x, uint64_t& y) {
            x = f2_add(v.x, x);
            y = f2_add(v.y, y);
        });
    };
    auto move_to_held = [&] {
        each_held([](ulonglong2& v, uint64_t& x, uint64_t& y) {
            v = make_ulonglong2(x, y);
            x = y = 0;
        });
    };
    const bool chained = (a.T + static_cast<int64_t>(gridDim.x) - 1) / gridDim.x > kChain * kTeams;
    if (chained) move_to_held();  // zeros
    int64_t t = r0 + team, chain_end = t + kChain * kTeams;
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch(t + k * kTeams, k);
    fetch_scales(t);
    int slot = 0, stage = 0;
    for (; t < r1; t += kTeams) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        uint32_t bytes[3][2];
#pragma unroll
        for (int k = 0; k < 3; ++k) bytes[k][0] = next[k][0], bytes[k][1] = next[k][1];
        fetch_scales(t + kTeams);
        auto read_dy = [&](int g, uint64_t (&v)[4]) {
            if (kGo == RLK_DTYPE_F32) {
                const uint4 lo = in[g] ? *place(stage, 2 * g) : uint4{}, hi = in[g] ? *place(stage, 2 * g + 1) : uint4{};
                v[0] = pair_of_words(lo.x, lo.y);
                v[1] = pair_of_words(lo.z, lo.w);
                v[2] = pair_of_words(hi.x, hi.y);
                v[3] = pair_of_words(hi.z, hi.w);
            } else {
                pairs_of(in[g] ? *place(stage, g) : uint4{}, v);
            }
        };
        auto read_saved = [&](int which, int k, int g, uint64_t (&v)[4]) {
            if (kSaved == RLK_SAVED_BF16) {
                pairs_of(in[g] ? *place(stage, k + g) : uint4{}, v);
            } else {
                const uint2 q = in[g] ? reinterpret_cast<const uint2*>(place(stage, k))[g] : uint2{};
                saved_decode8<kSaved>(q, saved_scale<kSaved>(bytes[which][g]), v);
            }
        };
        auto squares = [](const uint64_t (&v)[4]) {
            float s2[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                float lo, hi;
                f2_unpack(f2_mul(v[p], v[p]), lo, hi);
                s2[p] = __fadd_rn(lo, hi);
            }
            return __fadd_rn(__fadd_rn(s2[0], s2[1]), __fadd_rn(s2[2], s2[3]));
        };
        // the forward's tree over the squares of x and of the block, and up . x
        float sx[2], sb[2] = {0.0f, 0.0f};
        uint64_t dot = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint64_t x[4], dy[4], gam[4];
            read_saved(0, R::kX, g, x);
            read_dy(g, dy);
            pairs_of(gam_pre[g], gam);
            sx[g] = squares(x);
#pragma unroll
            for (int p = 0; p < 4; ++p) dot = f2_fma(f2_mul(dy[p], gam[p]), x[p], dot);
            if (post) {
                read_saved(1, R::kBlock, g, x);
                sb[g] = squares(x);
            }
        }
        auto across = [&](float s0, float s1) {  // both groups over the lanes, then one group and the other
            float q = __fadd_rn(odd ? s1 : s0, __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 1));
#pragma unroll
            for (int o = 2; o < 32; o <<= 1) q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, o));
            return __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, 1));
        };
        float d0, d1;
        f2_unpack(dot, d0, d1);
        float q = across(sx[0], sx[1]), qb = post ? across(sb[0], sb[1]) : 0.0f;
        float d = __fadd_rn(d0, d1);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
        if constexpr (kWarps > 1) {
            if (lane == 0) part[slot][team * kWarps + warp] = make_float4(q, d, qb, 0.0f);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kWarps) : "memory");
            float4 p[kWarps];
#pragma unroll
            for (int i = 0; i < kWarps; ++i) p[i] = part[slot][team * kWarps + i];
#pragma unroll
            for (int n = kWarps / 2; n >= 1; n >>= 1) {
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    p[i].x = __fadd_rn(p[2 * i].x, p[2 * i + 1].x);
                    p[i].y = __fadd_rn(p[2 * i].y, p[2 * i + 1].y);
                    p[i].z = __fadd_rn(p[2 * i].z, p[2 * i + 1].z);
                }
            }
            q = p[0].x;
            d = p[0].y;
            qb = p[0].z;
            slot ^= 1;  // a team's warps are never more than one sum apart
        }
        // a product with 1 / H is the quotient itself where H is a power of two
        auto rstd_of = [&](float sum) {
            return contract_rsqrt(__fadd_rn(pow2 ? __fmul_rn(sum, inv_h) : __fdiv_rn(sum, h), a.eps));
        };
        const float rstd = rstd_of(q);
        const float c = __fmul_rn(__fmul_rn(rstd, rstd), __fmul_rn(d, inv_h));
        const uint64_t rstd2 = f2_splat(rstd), neg_c2 = f2_splat(-c);
        const float rstd_b = post ? rstd_of(qb) : 1.0f;
        const uint64_t rstd_b2 = f2_splat(rstd_b);
        uint64_t v[2][4];  // the gradient that reaches the branch's norm, times gamma_post
        uint64_t dot_b = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t at = t * a.H + i0 + 256 * g;
            uint64_t dx[4];
            {
                uint64_t x[4], dy[4], gam[4], res[4] = {};
                read_saved(0, R::kX, g, x);
                read_dy(g, dy);
                pairs_of(gam_pre[g], gam);
                if (res_in_ring) pairs_of(in[g] ? *place(stage, R::kRes + g) : uint4{}, res);
                else if (a.grad_res && in[g]) load_grad(a.grad_res, a.gx_dtype, at, res);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    dx[p] = f2_fma(rstd2, f2_fma(x[p], neg_c2, f2_mul(dy[p], gam[p])), res[p]);
                    d_pre[g][p] = f2_fma(dy[p], f2_mul(x[p], rstd2), d_pre[g][p]);
                }
            }
            if (a.grad_residual && in[g]) {
                uint64_t o[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) o[p] = f2_mul(f2_splat(a.residual_scale), dx[p]);
                store_grad(a.grad_residual, a.gx_dtype, at, o);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) v[g][p] = f2_mul(f2_splat(a.block_scale), dx[p]);
            if (branch) {
                uint64_t b[4], gam[4];
                read_saved(1, R::kBlock, g, b);
                pairs_of(gam_post[g], gam);
                if (gated) {
                    uint64_t z[4], o[4];
                    read_saved(2, R::kGate, g, z);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        uint64_t gate, slope;
                        gate_of(a.gate_kind, z[p], gate, slope);
                        const uint64_t n = post ? f2_mul(f2_mul(b[p], rstd_b2), gam[p]) : b[p];
                        o[p] = f2_mul(f2_mul(v[g][p], n), slope);
                        v[g][p] = f2_mul(v[g][p], gate);
                    }
                    if (a.grad_gate && in[g]) store_grad(a.grad_gate, a.gx_dtype, at, o);
                }
                if (post) {
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        d_post[g][p] = f2_fma(v[g][p], f2_mul(b[p], rstd_b2), d_post[g][p]);
                        v[g][p] = f2_mul(v[g][p], gam[p]);
                        dot_b = f2_fma(v[g][p], b[p], dot_b);
                    }
                }
            }
            if (!post && a.grad_block && in[g]) store_grad(a.grad_block, a.gx_dtype, at, v[g]);
        }
        if (post && a.grad_block) {
            f2_unpack(dot_b, d0, d1);
            float k = __fadd_rn(d0, d1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, o));
            if constexpr (kWarps > 1) {
                if (lane == 0) part[slot][team * kWarps + warp].x = k;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kWarps) : "memory");
                float p[kWarps];
#pragma unroll
                for (int i = 0; i < kWarps; ++i) p[i] = part[slot][team * kWarps + i].x;
#pragma unroll
                for (int n = kWarps / 2; n >= 1; n >>= 1) {
#pragma unroll
                    for (int i = 0; i < n; ++i) p[i] = __fadd_rn(p[2 * i], p[2 * i + 1]);
                }
                k = p[0];
                slot ^= 1;
            }
            const uint64_t neg_k2 = f2_splat(-__fmul_rn(__fmul_rn(rstd_b, rstd_b), __fmul_rn(k, inv_h)));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint64_t b[4], o[4];
                read_saved(1, R::kBlock, g, b);
#pragma unroll
                for (int p = 0; p < 4; ++p) o[p] = f2_mul(rstd_b2, f2_fma(b[p], neg_k2, v[g][p]));
                if (in[g]) store_grad(a.grad_block, a.gx_dtype, t * a.H + i0 + 256 * g, o);
            }
        }
        fetch(t + kStages * kTeams, stage);  // everything in this stage has been used
        stage = stage + 1 < kStages ? stage + 1 : 0;
        if (chained && t + kTeams == chain_end) {
            add_held();
            move_to_held();
            chain_end += kChain * kTeams;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.grad_pre && !a.grad_post) return;
    if (chained) add_held();
    // the range's sums: the teams' in ascending order, by way of the ring once every warp has read
    // its last row out of it
    float* const teams = reinterpret_cast<float*>(ring);
    float* const out = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint64_t(&sum)[2][4] = which == 0 ? d_pre : d_post;
        if constexpr (kTeams == 1) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (in[g]) store_grad(out + which * a.H, RLK_DTYPE_F32, i0 + 256 * g, sum[g]);
        } else {
            __syncthreads();
#pragma unroll
            for (int g = 0; g < 2; ++g) store_grad(teams, RLK_DTYPE_F32, team * kWarps * 512 + i0 + 256 * g, sum[g]);
            __syncthreads();
            for (int i = threadIdx.x; i < a.H; i += kThreads) {
                float s = teams[i];
#pragma unroll
                for (int k = 1; k < kTeams; ++k) s = __fadd_rn(s, teams[k * kWarps * 512 + i]);
                out[which * a.H + i] = s;
            }
        }
    }
}

// The grad_gammas from the ranges' sums: 32 threads per feature, each taking every 32nd range in
// ascending order, then pairwise.
__global__ void __launch_bounds__(1024)
    k_gamma_sums(const float* parts, int ranges, int H, float* grad_pre, float* grad_post) {
    __shared__ float smem[32][33];
    const int c = threadIdx.x & 31, row = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    ptx::grid_dependency_wait();
    float s = 0.0f;
#pragma unroll 5
    for (int r = row; r < ranges; r += 32) s = __fadd_rn(s, parts[static_cast<int64_t>(r) * 2 * H + col]);
    smem[row][c] = s;
    __syncthreads();
    s = warp_sum(smem[c][row]);  // feature `row` of the CTA's 32, one range class per lane
    const int at = blockIdx.x * 32 + row;
    if (c == 0 && at < H && grad_pre) grad_pre[at] = s;
    if (c == 0 && at >= H && grad_post) grad_post[at - H] = s;
}

template <int kWarps, int kGo, int kSaved>
cudaError_t launch_row(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    constexpr size_t kSmem = Ring<kGo, kSaved>::kBytes + kHeldBytes;
    // once per device and kernel: the runtime keeps it, and asking each time costs the host 1 us
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k_block_norm_backward<kWarps, kGo, kSaved>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    k_block_norm_backward<kWarps, kGo, kSaved><<<blocks, kThreads, kSmem, stream>>>(a);
    return cudaGetLastError();
}

template <int kSaved>
cudaError_t launch_block_bwd(const BlockBwdArgs& a, cudaStream_t stream) {
    const int blocks = block_bwd_ranges(a.T);
    int warps = 1;
    while (warps * 512 < a.H) warps *= 2;
    cudaError_t e = cudaSuccess;
#define RLK_ROW(W)                                                                                  \
    case W:                                                                                         \
        e = a.go_dtype == RLK_DTYPE_F32 ? launch_row<W, RLK_DTYPE_F32, kSaved>(a, blocks, stream)   \
                                        : launch_row<W, RLK_DTYPE_BF16, kSaved>(a, blocks, stream); \
        break
    if (blocks > 0) switch (warps) {
        RLK_ROW(1);
        RLK_ROW(2);
        RLK_ROW(4);
        RLK_ROW(8);
        RLK_ROW(16);
        default: return cudaErrorInvalidValue;
    }
#undef RLK_ROW
    if (e != cudaSuccess || (!a.grad_pre && !a.grad_post)) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(2 * a.H / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_gamma_sums, static_cast<const float*>(a.parts), blocks, a.H, a.grad_pre, a.grad_post);
}

}  // namespace
}  // namespace rlk
