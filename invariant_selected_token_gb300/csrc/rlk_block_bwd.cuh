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
// The sums over all rows stay in registers, 32 a thread, which is why one CTA
// an SM takes many rows and why what is read of a row lies in shared memory and is
// decoded where it is used, up to three times, rather than held.
//
// What bounds it: with bf16 activations HBM (8191 x 8192, a block without a gate,
// 139 us, 0.87 of the copy rate; 4096 x 4096 with a gate 51 us, 0.79, a sigmoid one
// 56, 0.72).  From 8-bit checkpoints it is the instructions: 4096 x 4096, a sigmoid
// gate, int8, takes 61 us (0.54), e4m3 65 (0.51): 82 instructions a feature at 62 % of the issue slots,
// half of them in the FMA pipe, where a packed pair takes two cycles; 16 warps an SM
// and two barriers a row leave the rest idle.  Without a gate it is 45 us (0.56), without
// a branch 32 (0.71; fp32 grad_out); with fp32 gradients in and out, e4m3, 69 to 87
// (0.66 to 0.72).  64 rows are 7 us: one row's latency and the second launch's.
// Rows of fewer than 512 features leave lanes idle: 120000 x 192 takes 87 us without a gate in
// bf16, 160 with a sigmoid one from int8, 194 from e4m3 with fp32 gradients (floors 41, 45, 80).
#pragma once

#include <atomic>
#include <cstdint>

#include "rlk_block.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 512;  // of a CTA, one CTA per SM
constexpr int kMostStages = 4; // rows of a team in flight or at work
constexpr int kChain = 64;     // rows that a team adds one after the other before it starts a new sum

// What a call has of the branch: nothing (the RMSNorm's own backward), a block, or a block and a gate
// that multiplies as it is or through a sigmoid.
enum Form { kNoBranch = 0, kBlock = 1, kGated = 2, kSigmoid = 3 };

// 16-byte places of a thread's ring in one stage: 16 features of each tensor.
template <int kGo, int kSaved, int kForm, int kGx>
struct Ring {
    static constexpr int kSavedPlaces = kSaved == RLK_SAVED_BF16 ? 2 : 1;
    static constexpr int kX = kGo == RLK_DTYPE_F32 ? 4 : 2, kB = kX + kSavedPlaces;
    static constexpr int kGate = kB + (kForm >= kBlock ? kSavedPlaces : 0);
    static constexpr int kRes = kGate + (kForm >= kGated ? kSavedPlaces : 0);
    static constexpr size_t kPlaceBytes = size_t(kThreads) * sizeof(uint4);
    static constexpr size_t kHeldBytes = size_t(kThreads) * (kForm == kNoBranch ? 16 : 32) * sizeof(float);
    static constexpr size_t kRoom = 232448 - 2048;  // 227 KB less what is declared shared
    // beside two rows of sums the gammas do not fit into 128 registers: they are kept in shared memory
    // where there is room (4096 x 4096, gated, int8: 66 against 84 us, of which most went to spilled
    // registers, since the ring leaves next to no first-level cache for them)
    static constexpr int kGammaPlaces =
        kForm != kNoBranch && (2 * kRes + 4) * kPlaceBytes + kHeldBytes <= kRoom ? 4 : 0;
    // Where all of them do not fit twice beside the sums the residual's gradient is fetched into the
    // second-level cache with the rest and read from there while the sums over its row are formed, as it is in
    // fp32.  Read where it is needed, that cost 64 us instead of 53 (4096 x 4096, gated, bf16); for those
    // that fit, early reads cost 155 instead of 138 us (8191 x 8192, bf16).
    static constexpr bool kHasRes =
        kGx == RLK_DTYPE_BF16 && (2 * (kRes + 2) + kGammaPlaces) * kPlaceBytes + kHeldBytes <= kRoom;
    static constexpr int kPlaces = kRes + (kHasRes ? 2 : 0);
    static constexpr size_t kStageBytes = kPlaces * kPlaceBytes;
    static_assert(2 * kStageBytes + kGammaPlaces * kPlaceBytes + kHeldBytes <= kRoom, "a row flies while another is worked on");
    static constexpr int stages(bool chained) {
        const int n = int((kRoom - kGammaPlaces * kPlaceBytes - (chained ? kHeldBytes : 0)) / kStageBytes);
        return n < kMostStages ? n : kMostStages;
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// All but the newest n groups of copies have landed.
__device__ __forceinline__ void wait_copies(int n) {
    if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

__device__ __forceinline__ void pairs_of_f32(uint4 lo, uint4 hi, uint64_t (&v)[4]) {
    v[0] = f2_pack(__uint_as_float(lo.x), __uint_as_float(lo.y));
    v[1] = f2_pack(__uint_as_float(lo.z), __uint_as_float(lo.w));
    v[2] = f2_pack(__uint_as_float(hi.x), __uint_as_float(hi.y));
    v[3] = f2_pack(__uint_as_float(hi.z), __uint_as_float(hi.w));
}
// fp32 features lie 32 bytes a lane.  A warp copies them as they lie in memory, 512 bytes an
// instruction, into two places of its own, 64 vectors in a row, of which every other 8 have their
// neighbours exchanged: so the 8 lanes that a shared-memory access serves at a time find one half
// of their features in 8 different places.
__device__ __forceinline__ int f32_place(int vec) { return vec ^ ((vec >> 3) & 1); }

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

__device__ __forceinline__ void store_f32(float* to, const uint64_t (&v)[4]) {
    float e[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) f2_unpack(v[p], e[2 * p], e[2 * p + 1]);
    reinterpret_cast<float4*>(to)[0] = make_float4(e[0], e[1], e[2], e[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(e[4], e[5], e[6], e[7]);
}
// 8 features of a gradient at element i.  Called by whole warps; a pair of lanes is in or out together.
template <int kDtype>
__device__ __forceinline__ void store_grad(void* base, int64_t i, bool in, const uint64_t (&v)[4]) {
    if (kDtype == RLK_DTYPE_F32) {
        // even lanes hand their last four features over for the odd ones' first four, so that a lane
        // pair stores whole sectors
        const bool odd = threadIdx.x & 1;
        const uint64_t r0 = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[2], 1);
        const uint64_t r1 = __shfl_xor_sync(0xffffffffu, odd ? v[1] : v[3], 1);
        float e[8];
        f2_unpack(odd ? r0 : v[0], e[0], e[1]);
        f2_unpack(odd ? r1 : v[1], e[2], e[3]);
        f2_unpack(odd ? v[2] : r0, e[4], e[5]);
        f2_unpack(odd ? v[3] : r1, e[6], e[7]);
        if (in) {
            float* const to = static_cast<float*>(base) + i - (odd ? 4 : 0);
            *reinterpret_cast<float4*>(to) = make_float4(e[0], e[1], e[2], e[3]);
            *reinterpret_cast<float4*>(to + 8) = make_float4(e[4], e[5], e[6], e[7]);
        }
    } else if (in) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = words_of(v);
    }
}

// 128 registers a thread hold two sums and a row's work, but for some instances with a gate: for rows of
// one warp and of 16 warps up to 40 bytes are spilled, for the widths between none.
//
// A team of kWarps warps (a power of two) takes a row, a CTA's teams every kTeams-th row of its
// range.  A thread copies its own features of the next rows into its own places of a ring of shared
// memory, which needs no barrier; the copies fly while the current row is reduced.  Places of features
// behind the row's end hold zeros.
template <int kWarps, int kGo, int kSaved, int kForm, int kGx>
__global__ void __launch_bounds__(kThreads, 1) k_block_norm_backward(const BlockBwdArgs a, const int stages) {
    using R = Ring<kGo, kSaved, kForm, kGx>;
    constexpr int kTeams = kThreads / 32 / kWarps;
    constexpr bool kPlain = kSaved == RLK_SAVED_BF16;
    static_assert(kWarps == 1 || kTeams <= 15, "a named barrier (1 .. 15) per team");
    extern __shared__ uint4 ring[];  // [stage][place][thread]
    __shared__ __align__(16) float4 part[2][kThreads / 32];
    ptx::grid_dependents_launch();
    const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * kWarps);
    const int warp_of_cta = threadIdx.x >> 5, warp = warp_of_cta % kWarps;
    const int i0 = 512 * warp + 8 * lane;  // and i0 + 256
    const int f32_left = a.H - 512 * warp - 4 * lane;  // from this lane's first vector of fp32 features on
    const bool in[2] = {i0 < a.H, i0 + 256 < a.H};
    // rows stay below 2^31 - 2^20, and a team looks at most 64 rows past the last
    const int r0 = static_cast<int>(static_cast<int64_t>(a.T) * blockIdx.x / gridDim.x);
    const int r1 = static_cast<int>(static_cast<int64_t>(a.T) * (blockIdx.x + 1) / gridDim.x);
    const bool pow2 = (a.H & (a.H - 1)) == 0;
    const float inv_h = __fdiv_rn(1.0f, static_cast<float>(a.H));
    const bool post = kForm != kNoBranch && a.gamma_post != nullptr;
    const bool res_in_ring = R::kHasRes && a.grad_res;
    const bool res_early = !R::kHasRes && a.grad_res;
    constexpr int kResVecs = kGx == RLK_DTYPE_F32 ? 2 : 1;  // of 16 bytes, 8 features
    auto res_at = [&](int64_t i) {
        return reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.grad_res) + i * (2 * kResVecs));
    };
    if (512 * (warp + 1) > a.H) {  // features behind the row's end are read as zeros
        for (int k = 0; k < stages * R::kPlaces; ++k) {
            // a warp's fp32 vectors of a group, 64 in a row over two places, or a thread's own place
            const int r = k % R::kPlaces, half = r & 1;
            const int at = kGo == RLK_DTYPE_F32 && r < R::kX ? (k - half) * kThreads + 64 * warp_of_cta + 32 * half + lane
                                                             : k * kThreads + threadIdx.x;
            ring[at] = make_uint4(0u, 0u, 0u, 0u);
        }
        __syncwarp();
    }
    const uint32_t mine = ptx::smem_addr(ring + threadIdx.x);
    auto place = [&](int stage, int k) { return ring + (stage * R::kPlaces + k) * kThreads + threadIdx.x; };

    // i: this thread's first element of row t.  The distance between a team's rows is kept where there are
    // registers to spare (32771 x 1024 from e4m3: 45 against 49 us).
    const int64_t step = static_cast<int64_t>(kTeams) * a.H;
    auto ahead = [&](int rows) { return kForm == kNoBranch ? rows * step : static_cast<int64_t>(rows * kTeams) * a.H; };
    auto fetch_saved = [&](const SavedIn& s, int64_t i, uint32_t to, int g) {
        if (kPlain) copy16(to + g * (kThreads * 16), static_cast<const uint16_t*>(s.data) + i + 256 * g);
        else copy8(to + g * 8, static_cast<const uint8_t*>(s.data) + i + 256 * g);
    };
    auto fetch = [&](int t, int64_t i, int stage) {
        if (t < r1) {
            const uint32_t to = mine + static_cast<uint32_t>(stage) * uint32_t(R::kStageBytes);
            constexpr uint32_t kStep = kThreads * 16;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (kGo == RLK_DTYPE_F32) {
                    // the warp's 64 vectors of this group, two places; this lane's share are lane and lane + 32
                    const float* from = static_cast<const float*>(a.grad_out) + i + 256 * g - 4 * lane;
                    const uint32_t at = to + 2 * g * kStep + (32 * warp_of_cta + f32_place(lane) - lane) * 16;
                    if (f32_left > 256 * g) copy16(at, from);
                    if (f32_left > 256 * g + 128) copy16(at + 32 * 16, from + 128);
                }
                if (!in[g]) continue;
                if (kGo == RLK_DTYPE_BF16) copy16(to + g * kStep, static_cast<const uint16_t*>(a.grad_out) + i + 256 * g);
                fetch_saved(a.x, i, to + R::kX * kStep, g);
                if constexpr (kForm >= kBlock) fetch_saved(a.block, i, to + R::kB * kStep, g);
                if constexpr (kForm >= kGated) fetch_saved(a.gate, i, to + R::kGate * kStep, g);
                if (res_in_ring) copy16(to + (R::kRes + g) * kStep, static_cast<const uint16_t*>(a.grad_res) + i + 256 * g);
                if (res_early) prefetch_l2(res_at(i + 256 * g));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // the bytes of this thread's blocks of 32 features, a row ahead
    uint32_t next[3][2] = {};
    auto fetch_scales = [&](int t, int64_t i) {
        if constexpr (!kPlain) {
            if (t >= r1) return;
            const int64_t k = i >> 5;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!in[g]) continue;
                next[0][g] = a.x.scales[k + 8 * g];
                if constexpr (kForm >= kBlock) next[1][g] = a.block.scales[k + 8 * g];
                if constexpr (kForm >= kGated) next[2][g] = a.gate.scales[k + 8 * g];
            }
        }
    };
    uint4 gam[4] = {};  // pre, post
    uint4* const gammas = ring + stages * R::kPlaces * kThreads + threadIdx.x;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        if (in[g]) gam[g] = *reinterpret_cast<const uint4*>(a.gamma_pre + i0 + 256 * g);
        if (in[g] && post) gam[2 + g] = *reinterpret_cast<const uint4*>(a.gamma_post + i0 + 256 * g);
    }
    if constexpr (R::kGammaPlaces != 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) gammas[k * kThreads] = gam[k];
    }
    auto read_gamma = [&](int k, uint64_t (&v)[4]) {
        if constexpr (R::kGammaPlaces != 0) pairs_of(gammas[k * kThreads], v);
        else pairs_of(gam[k], v);
    };
    uint64_t d_pre[2][4] = {}, d_post[2][4] = {};
    ulonglong2* const held = reinterpret_cast<ulonglong2*>(gammas + R::kGammaPlaces * kThreads);
    auto each_held = [&](auto fn) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            fn(held[k * kThreads], d_pre[k >> 1][2 * (k & 1)], d_pre[k >> 1][2 * (k & 1) + 1]);
            if constexpr (kForm != kNoBranch)
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
    const bool chained = block_bwd_chained(a.T, gridDim.x, kTeams);
    if (chained) move_to_held();  // zeros
    int t = r0 + team, chain_end = t + kChain * kTeams;
    int64_t i = static_cast<int64_t>(t) * a.H + i0;
    for (int k = 0; k < stages; ++k) fetch(t + k * kTeams, i + ahead(k), k);
    fetch_scales(t, i);
    int slot = 0, stage = 0;
    for (; t < r1; t += kTeams, i += ahead(1)) {
        wait_copies(stages - 1);
        if (kGo == RLK_DTYPE_F32) __syncwarp();  // the lanes of a warp share what they copied
        float scale[3][2];
        if constexpr (!kPlain) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
                for (int g = 0; g < 2; ++g) scale[k][g] = saved_scale<kSaved>(next[k][g]);
            fetch_scales(t + kTeams, i + ahead(1));
        }
        auto read_dy = [&](int g, uint64_t (&v)[4]) {
            if constexpr (kGo == RLK_DTYPE_F32) {
                const uint4* const own = place(stage, 2 * g) + 32 * warp_of_cta - lane;  // the warp's 64 vectors
                const int at = f32_place(2 * lane);
                pairs_of_f32(own[at], own[at ^ 1], v);
            } else {
                pairs_of(*place(stage, g), v);
            }
        };
        auto read_saved = [&](int which, int k, int g, uint64_t (&v)[4]) {
            if constexpr (kPlain) pairs_of(*place(stage, k + g), v);
            else saved_decode8<kSaved>(reinterpret_cast<const uint2*>(place(stage, k))[g], scale[which][g], v);
        };
        // the forward's tree over the squares of x and of the block, and up . x
        float sx[2], sb[2] = {0.0f, 0.0f}, d0, d1;
        uint64_t dot = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint64_t x[4], dy[4], gam[4];
            read_saved(0, R::kX, g, x);
            read_dy(g, dy);
            read_gamma(g, gam);
            sx[g] = squares_of(x);
#pragma unroll
            for (int p = 0; p < 4; ++p) dot = f2_fma(f2_mul(dy[p], gam[p]), x[p], dot);
            if (post) {
                read_saved(1, R::kB, g, x);
                sb[g] = squares_of(x);
            }
        }
        uint4 early[2][kResVecs] = {};  // on their way while the sums are formed
        if (res_early) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int k = 0; k < kResVecs; ++k)
                    if (in[g]) early[g][k] = res_at(i + 256 * g)[k];
        }
        f2_unpack(dot, d0, d1);
        float sums = warp_sums<kForm != kNoBranch>(sx, sb, __fadd_rn(d0, d1));
        float d;
        if constexpr (kWarps == 1) {
            d = __shfl_sync(0xffffffffu, sums, 4);
            // nothing read so far is kept, as behind the other teams' barrier: there are no registers for it
            // (60000 x 512, gated, int8: 75 us instead of 95)
            asm volatile("" ::: "memory");
        } else {
            if (lane < 6 && !(lane & 1)) reinterpret_cast<float*>(&part[slot][team * kWarps + warp])[lane >> 1] = sums;
            team_barrier<kWarps>(team);
            sums = team_sums<kWarps>(&part[slot][team * kWarps]);
            d = kWarps <= 8 ? __shfl_sync(0xffffffffu, sums, (2 * kWarps) & 31) : team_sum<kWarps>(&part[slot][team * kWarps], 2);
        }
        // a product with 1 / H is the quotient itself where H is a power of two
        const float root = contract_rsqrt(__fadd_rn(pow2 ? __fmul_rn(sums, inv_h) : __fdiv_rn(sums, static_cast<float>(a.H)), a.eps));
        const float rstd = __shfl_sync(0xffffffffu, root, 0);
        const float rstd_b = post ? __shfl_sync(0xffffffffu, root, kWarps == 1 ? 2 : kWarps) : 1.0f;
        const float c = __fmul_rn(__fmul_rn(rstd, rstd), __fmul_rn(d, inv_h));
        const uint64_t rstd2 = f2_splat(rstd), neg_c2 = f2_splat(-c), rstd_b2 = f2_splat(rstd_b);
        uint64_t v[2][4];  // the gradient that reaches the branch's norm, times gamma_post
        uint64_t dot_b = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t at = i + 256 * g;
            uint64_t dx[4];
            {
                uint64_t x[4], dy[4], gam[4], res[4] = {};
                read_saved(0, R::kX, g, x);
                read_dy(g, dy);
                read_gamma(g, gam);
                if (res_in_ring) pairs_of(*place(stage, R::kRes + g), res);
                else if (res_early && kResVecs == 1) pairs_of(early[g][0], res);
                else if (res_early) pairs_of_f32(early[g][0], early[g][kResVecs - 1], res);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    dx[p] = f2_fma(rstd2, f2_fma(x[p], neg_c2, f2_mul(dy[p], gam[p])), res[p]);
                    d_pre[g][p] = f2_fma(dy[p], f2_mul(x[p], rstd2), d_pre[g][p]);
                }
            }
            if (a.grad_residual) {
                uint64_t o[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) o[p] = f2_mul(f2_splat(a.residual_scale), dx[p]);
                store_grad<kGx>(a.grad_residual, at, in[g], o);
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) v[g][p] = f2_mul(f2_splat(a.block_scale), dx[p]);
            if constexpr (kForm != kNoBranch) {
                uint64_t b[4], gam[4];
                read_saved(1, R::kB, g, b);
                read_gamma(2 + g, gam);
                if constexpr (kForm >= kGated) {
                    uint64_t z[4], o[4];
                    read_saved(2, R::kGate, g, z);
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const uint64_t n = post ? f2_mul(f2_mul(b[p], rstd_b2), gam[p]) : b[p];
                        o[p] = f2_mul(v[g][p], n);
                        if constexpr (kForm == kSigmoid) {
                            uint64_t e;
                            sigmoid_of(z[p], e, z[p]);
                            o[p] = f2_mul(o[p], f2_mul(f2_mul(e, z[p]), z[p]));
                        }
                        v[g][p] = f2_mul(v[g][p], z[p]);
                    }
                    if (a.grad_gate) store_grad<kGx>(a.grad_gate, at, in[g], o);
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
            if (!post && a.grad_block) store_grad<kGx>(a.grad_block, at, in[g], v[g]);
        }
        if (post && a.grad_block) {
            f2_unpack(dot_b, d0, d1);
            float k = __fadd_rn(d0, d1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, o));
            if constexpr (kWarps > 1) {
                // a place of its own in this row's slot; the next row takes the other one
                if (lane == 0) part[slot][team * kWarps + warp].w = k;
                team_barrier<kWarps>(team);
                k = team_sum<kWarps>(&part[slot][team * kWarps], 3);
            } else {
                asm volatile("" ::: "memory");  // as above
            }
            const uint64_t neg_k2 = f2_splat(-__fmul_rn(__fmul_rn(rstd_b, rstd_b), __fmul_rn(k, inv_h)));
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint64_t b[4], o[4];
                read_saved(1, R::kB, g, b);
#pragma unroll
                for (int p = 0; p < 4; ++p) o[p] = f2_mul(rstd_b2, f2_fma(b[p], neg_k2, v[g][p]));
                store_grad<kGx>(a.grad_block, i + 256 * g, in[g], o);
            }
        }
        slot ^= 1;  // a team's warps are never more than one row apart
        if (kGo == RLK_DTYPE_F32) __syncwarp();
        fetch(t + stages * kTeams, i + ahead(stages), stage);  // everything in this stage has been used
        stage = stage + 1 < stages ? stage + 1 : 0;
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
    for (int which = 0; which < (kForm == kNoBranch ? 1 : 2); ++which) {
        uint64_t(&sum)[2][4] = which == 0 ? d_pre : d_post;
        if constexpr (kTeams == 1) {
#pragma unroll
            for (int g = 0; g < 2; ++g)
                if (in[g]) store_f32(out + which * a.H + i0 + 256 * g, sum[g]);
        } else {
            __syncthreads();
#pragma unroll
            for (int g = 0; g < 2; ++g) store_f32(teams + team * kWarps * 512 + i0 + 256 * g, sum[g]);
            __syncthreads();
            for (int k = threadIdx.x; k < a.H; k += kThreads) {
                float s = teams[k];
#pragma unroll
                for (int n = 1; n < kTeams; ++n) s = __fadd_rn(s, teams[n * kWarps * 512 + k]);
                out[which * a.H + k] = s;
            }
        }
    }
}

template <int kWarps, int kGo, int kSaved, int kForm, int kGx>
cudaError_t launch_gx(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    using R = Ring<kGo, kSaved, kForm, kGx>;
    const bool chained = block_bwd_chained(a.T, blocks, kThreads / 32 / kWarps);
    const int stages = R::stages(chained);
    // once per device and kernel: the runtime keeps it, and asking each time costs the host 1 us
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k_block_norm_backward<kWarps, kGo, kSaved, kForm, kGx>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(R::kRoom));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const size_t smem = stages * R::kStageBytes + R::kGammaPlaces * R::kPlaceBytes + (chained ? R::kHeldBytes : 0);
    k_block_norm_backward<kWarps, kGo, kSaved, kForm, kGx><<<blocks, kThreads, smem, stream>>>(a, stages);
    return cudaGetLastError();
}

template <int kWarps, int kGo, int kSaved, int kForm>
cudaError_t launch_form(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    return a.gx_dtype == RLK_DTYPE_F32 ? launch_gx<kWarps, kGo, kSaved, kForm, RLK_DTYPE_F32>(a, blocks, stream)
                                       : launch_gx<kWarps, kGo, kSaved, kForm, RLK_DTYPE_BF16>(a, blocks, stream);
}

template <int kWarps, int kGo, int kSaved>
cudaError_t launch_row(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    if (!a.block.data) return launch_form<kWarps, kGo, kSaved, kNoBranch>(a, blocks, stream);
    if (!a.gate.data) return launch_form<kWarps, kGo, kSaved, kBlock>(a, blocks, stream);
    return a.gate_kind == RLK_GATE_SIGMOID ? launch_form<kWarps, kGo, kSaved, kSigmoid>(a, blocks, stream)
                                           : launch_form<kWarps, kGo, kSaved, kGated>(a, blocks, stream);
}

// grad_out's types apart, a translation unit each
template <int kGo, int kSaved>
cudaError_t launch_rows(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    int warps = 1;
    while (warps * 512 < a.H) warps *= 2;
    switch (warps) {
        case 1: return launch_row<1, kGo, kSaved>(a, blocks, stream);
        case 2: return launch_row<2, kGo, kSaved>(a, blocks, stream);
        case 4: return launch_row<4, kGo, kSaved>(a, blocks, stream);
        case 8: return launch_row<8, kGo, kSaved>(a, blocks, stream);
        case 16: return launch_row<16, kGo, kSaved>(a, blocks, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace
}  // namespace rlk
