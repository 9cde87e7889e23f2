// The norms before and after a block, its gate and the residual stream's
// scales in one pass.  Per row, in fp32,
//
//   n   = RN(RN(b rstd(b)) gamma_post)        (b itself without gamma_post)
//   x'  = bf16_RN(fma(rs, r, bs (n gate)))
//   out = bf16_RN(RN(RN(x' rstd(x')) gamma_pre))
//
// with rstd by the strict RMSNorm's tree and rsqrt, so that out has the bits of
// rlk_rmsnorm on x'.  The checkpoints for the backward are formed from the same
// registers.
//
// Element i = 512 w + 256 g + 8 l + j is warp w's lane l's j-th value of its
// column group g: a lane reads 16 contiguous bytes, four lanes hold a
// checkpoint's block of 32, and the tree's levels fall as in the RMSNorm: over j
// in the lane, over l across lanes, over the two groups, then over the warps.
// 16 features a thread keep a row in registers between the two norms, so that it
// is read once.
//
// What bounds it: HBM.  16384 x 4096 takes 82 us (0.98 of the copy rate on the
// bytes it has to move), 8191 x 8192 92 us (0.87), 4096 x 4096 24 (0.83) and with a
// sigmoid gate 32 (0.79, start and tail of a short launch; 0.92 at 16384 rows); storing three
// checkpoints 40 of either kind (0.83; 71 % of the issue slots, 61 instructions a
// feature, a third of them for codes and scales), without a gate two 30 (0.83).  8 rows are 2.5 us of
// latency: two loads and two sums over a row, one after the other.
#include <cstdint>

#include "rlk_block.cuh"

namespace rlk {
namespace {

// Teams of one and two warps share a CTA of 256 threads: with 128 32768 x 1024 takes 53 us instead of 47, with
// three checkpoints and their restoring 147 instead of 122, 60000 x 512 the same within 2 %; two teams of four
// warps (16384 x 2048) take 47 instead of 43 for one.
constexpr int cta_threads(int warps) { return warps <= 2 ? 256 : 32 * warps; }

template <int kSaved>
__device__ __forceinline__ void save_group(const SavedOut& to, uint4 x, int64_t at, bool in) {
    uint32_t m = amax8(x);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t byte = saved_byte<kSaved>(m);
    const uint2 codes = saved_encode8<kSaved>(x, m, byte);
    if (!in) return;
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(to.codes) + at) = codes;
    if (!(threadIdx.x & 3)) to.scales[at >> 5] = static_cast<uint8_t>(byte);
}

// A team of kWarps warps per row.
template <int kWarps, int kSaved>
__global__ void __launch_bounds__(cta_threads(kWarps)) k_block_norm(const BlockNormArgs a) {
    constexpr int kTeams = cta_threads(kWarps) / (32 * kWarps);
    __shared__ float part[kTeams][2][kWarps];  // [team][slot][warp]
    const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * kWarps);
    const int warp = (threadIdx.x >> 5) % kWarps;
    const int i0 = 512 * warp + 8 * lane;  // and i0 + 256
    const bool in[2] = {i0 < a.H, i0 + 256 < a.H};
    const int odd = lane & 1;
    const bool pow2 = (a.H & (a.H - 1)) == 0;
    const float h = static_cast<float>(a.H), inv_h = __fdiv_rn(1.0f, h);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;

    // rstd of the row whose 16 features are v: the contract's tree
    auto rstd_of = [&](const uint64_t (&v)[2][4], int slot) {
        const float s0 = squares_of(v[0]), s1 = squares_of(v[1]);
        // even lanes go on with the first group, odd ones with the second
        float q = __fadd_rn(odd ? s1 : s0, __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 1));
#pragma unroll
        for (int o = 2; o < 32; o <<= 1) q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, o));
        q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, 1));
        if constexpr (kWarps > 1) {
            // two slots alternate: a team's warps are never more than one sum apart
            if (lane == 0) part[team][slot][warp] = q;
            team_barrier<kWarps>(team);
            q = part[team][slot][lane & (kWarps - 1)];
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, o));
        }
        // a product with 1 / H is the quotient itself where H is a power of two
        return contract_rsqrt(__fadd_rn(pow2 ? __fmul_rn(q, inv_h) : __fdiv_rn(q, h), a.eps));
    };
    auto load = [&](const uint16_t* base, int64_t row, uint4 (&w)[2]) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
            w[g] = in[g] ? *reinterpret_cast<const uint4*>(base + row + i0 + 256 * g) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto pairs = [](const uint4 (&w)[2], uint64_t (&v)[2][4]) {
        pairs_of(w[0], v[0]);
        pairs_of(w[1], v[1]);
    };

    int slot = 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTeams + team; t < a.T; t += stride) {
        const int64_t row = t * a.H;
        uint4 wb[2], wr[2], wg[2];
        load(a.block, row, wb);
        load(a.residual, row, wr);
        if (a.gate) load(a.gate, row, wg);
        if constexpr (kSaved != RLK_SAVED_BF16) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (a.saved_block.codes) save_group<kSaved>(a.saved_block, wb[g], row + i0 + 256 * g, in[g]);
                if (a.saved_gate.codes) save_group<kSaved>(a.saved_gate, wg[g], row + i0 + 256 * g, in[g]);
            }
        }
        uint64_t n[2][4];
        pairs(wb, n);
        if (a.gamma_post) {
            uint4 w[2];
            load(a.gamma_post, 0, w);  // on its way while the sum is formed
            const uint64_t rstd = f2_splat(rstd_of(n, slot));
            slot ^= 1;
            uint64_t gam[2][4];
            pairs(w, gam);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int p = 0; p < 4; ++p) n[g][p] = f2_mul(f2_mul(n[g][p], rstd), gam[g][p]);
        }
        if (a.gate) {
            uint64_t z[2][4];
            pairs(wg, z);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    if (a.gate_kind == RLK_GATE_SIGMOID) {
                        uint64_t e, r;
                        sigmoid_of(z[g][p], e, r);
                        z[g][p] = r;
                    }
                    n[g][p] = f2_mul(n[g][p], z[g][p]);
                }
        }
        uint64_t x[2][4];
        pairs(wr, x);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                o[p] = pack_bf16x2(f2_fma(f2_splat(a.residual_scale), x[g][p], f2_mul(n[g][p], f2_splat(a.block_scale))));
                x[g][p] = unpack_bf16x2(o[p]);  // the norm's input is the stream as it is stored
            }
            const uint4 w = make_uint4(o[0], o[1], o[2], o[3]);
            const int64_t at = row + i0 + 256 * g;
            if (in[g]) *reinterpret_cast<uint4*>(a.residual_out + at) = w;
            if constexpr (kSaved != RLK_SAVED_BF16) save_group<kSaved>(a.saved_x, w, at, in[g]);
        }
        uint4 w[2];
        load(a.gamma_pre, 0, w);
        const uint64_t rstd = f2_splat(rstd_of(x, slot));
        slot ^= 1;
        uint64_t gam[2][4];
        pairs(w, gam);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) o[p] = pack_bf16x2(f2_mul(f2_mul(x[g][p], rstd), gam[g][p]));
            if (in[g]) *reinterpret_cast<uint4*>(a.out + row + i0 + 256 * g) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <int kWarps, int kSaved>
cudaError_t launch(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
    constexpr int kTeams = cta_threads(kWarps) / (32 * kWarps);
    int64_t blocks = (static_cast<int64_t>(a.T) + kTeams - 1) / kTeams;
    // several rows a team only from 64 CTAs an SM on: with 32 16384 x 4096 takes 83.3 instead of 82.5 us, 8191 x
    // 8192 with three int8 checkpoints and their restoring 253 instead of 246, without them 91 instead of 92
    if (blocks > static_cast<int64_t>(num_sms) * 64) blocks = static_cast<int64_t>(num_sms) * 64;
    k_block_norm<kWarps, kSaved><<<static_cast<int>(blocks), cta_threads(kWarps), 0, stream>>>(a);
    return cudaGetLastError();
}

template <int kSaved>
cudaError_t launch_saved(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
    int warps = 1;
    while (warps * 512 < a.H) warps *= 2;
    switch (warps) {
        case 1: return launch<1, kSaved>(a, num_sms, stream);
        case 2: return launch<2, kSaved>(a, num_sms, stream);
        case 4: return launch<4, kSaved>(a, num_sms, stream);
        case 8: return launch<8, kSaved>(a, num_sms, stream);
        case 16: return launch<16, kSaved>(a, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
    switch (a.saved_format) {
        case RLK_SAVED_BF16: return launch_saved<RLK_SAVED_BF16>(a, num_sms, stream);
        case RLK_SAVED_INT8: return launch_saved<RLK_SAVED_INT8>(a, num_sms, stream);
        default: return launch_saved<RLK_SAVED_E4M3>(a, num_sms, stream);
    }
}

}  // namespace rlk
