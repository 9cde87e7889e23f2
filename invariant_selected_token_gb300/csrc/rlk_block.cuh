// Shared by the block norms, the 8-bit activation checkpoints and the draft
// verification: the launch interface between the host dispatcher and their
// kernels, and the device arithmetic of the checkpoints.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/rlk.h"
#include "rlk_contract.cuh"

namespace rlk {

// ---------------------------------------------------------------- launches
// A [T][H] activation: a bf16 tensor, or 8-bit codes with a byte per 32 features.
struct SavedIn {
    const void* data;
    const uint8_t* scales;
};
struct SavedOut {
    void* codes;
    uint8_t* scales;
};

cudaError_t launch_act_quantize(const uint16_t* x, int format, int64_t n, SavedOut out, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_act_dequantize(SavedIn in, int format, int64_t n, uint16_t* out, int num_sms,
                                  cudaStream_t stream);

struct BlockNormArgs {
    const uint16_t* block;       // bf16 [T][H]
    const uint16_t* gamma_post;  // bf16 [H] or nullptr
    const uint16_t* gate;        // bf16 [T][H] or nullptr
    const uint16_t* residual;    // bf16 [T][H]
    const uint16_t* gamma_pre;   // bf16 [H]
    uint16_t* out;               // bf16 [T][H]
    uint16_t* residual_out;      // bf16 [T][H]
    SavedOut saved_x, saved_block, saved_gate;  // codes nullptr where not wanted
    float residual_scale, block_scale, eps;
    int gate_kind, saved_format;
    int T, H;
};
cudaError_t launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t stream);

struct BlockBwdArgs {
    const void* grad_out;        // [T][H] of go_dtype
    const void* grad_res;        // [T][H] of gx_dtype, or nullptr
    SavedIn x, block, gate;      // block.data nullptr: there is no branch but a plain sum
    const uint16_t* gamma_post;  // bf16 [H] or nullptr
    const uint16_t* gamma_pre;   // bf16 [H]
    void* grad_residual;         // [T][H] of gx_dtype, each or nullptr
    void* grad_block;
    void* grad_gate;
    float* grad_pre;             // [H] or nullptr
    float* grad_post;            // [H] or nullptr
    float* parts;                // workspace [ranges][2][H]
    float residual_scale, block_scale, eps;
    int gate_kind, go_dtype, gx_dtype;
    int T, H;
};
// Ranges of rows whose grad_gamma sums are formed apart, a CTA per SM each.
constexpr int kBlockBwdRanges = 152;
inline int block_bwd_ranges(int64_t T) { return T < kBlockBwdRanges ? static_cast<int>(T) : kBlockBwdRanges; }
// Whether a team has more than one chain of 64 rows.
__host__ __device__ inline bool block_bwd_chained(int64_t T, int64_t blocks, int teams) {
    return (T + blocks - 1) / blocks > 64 * int64_t(teams);
}
cudaError_t launch_block_bwd(const BlockBwdArgs& a, int format, cudaStream_t stream);
// a translation unit for each kind of saved activation and each type of grad_out
cudaError_t launch_block_bwd_bf16_f32(const BlockBwdArgs& a, int blocks, cudaStream_t stream);
cudaError_t launch_block_bwd_bf16_bf16(const BlockBwdArgs& a, int blocks, cudaStream_t stream);
cudaError_t launch_block_bwd_int8_f32(const BlockBwdArgs& a, int blocks, cudaStream_t stream);
cudaError_t launch_block_bwd_int8_bf16(const BlockBwdArgs& a, int blocks, cudaStream_t stream);
cudaError_t launch_block_bwd_e4m3_f32(const BlockBwdArgs& a, int blocks, cudaStream_t stream);
cudaError_t launch_block_bwd_e4m3_bf16(const BlockBwdArgs& a, int blocks, cudaStream_t stream);

struct VerifyArgs {
    const void* target;          // [rows][ld_target]
    const void* draft;           // [n_draft][ld_draft] or nullptr
    const float* draft_lse;      // [n_draft] or nullptr
    const int32_t* tokens;       // [n_draft]
    const float* uniforms;       // [n_draft]
    const float* noise;          // [n_seqs][ld_noise]
    const int32_t* offsets;      // [n_seqs + 1]
    const uint8_t* active;       // [n_seqs] or nullptr
    const float2* partials;      // [n_draft + n_seqs][n_tiles]: the rows' tile pairs
    int n_tiles, depth;          // of the tile tree: leaves, and ceil(log2) of them
    int64_t ld_target, ld_draft, ld_noise;
    int target_dtype, draft_dtype;
    int n_draft, n_seqs, V;
    bool fetch_noise;            // ahead, into the second-level cache
    int32_t* out_accepted;
    int32_t* out_tokens;
    float* out_logprob;
    int32_t* status;
};
cudaError_t launch_draft_verify(const VerifyArgs& a, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- bf16 pairs
__device__ __forceinline__ uint32_t pack_bf16x2(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint64_t unpack_bf16x2(uint32_t w) {
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void pairs_of(uint4 w, uint64_t (&v)[4]) {
    v[0] = unpack_bf16x2(w.x);
    v[1] = unpack_bf16x2(w.y);
    v[2] = unpack_bf16x2(w.z);
    v[3] = unpack_bf16x2(w.w);
}
__device__ __forceinline__ uint4 words_of(const uint64_t (&v)[4]) {
    return make_uint4(pack_bf16x2(v[0]), pack_bf16x2(v[1]), pack_bf16x2(v[2]), pack_bf16x2(v[3]));
}
// The contract's tree over the squares of 8 features.
__device__ __forceinline__ float squares_of(const uint64_t (&v)[4]) {
    float s2[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        float lo, hi;
        f2_unpack(f2_mul(v[p], v[p]), lo, hi);
        s2[p] = __fadd_rn(lo, hi);
    }
    return __fadd_rn(__fadd_rn(s2[0], s2[1]), __fadd_rn(s2[2], s2[3]));
}

// e^-z and the sigmoid 1 / (1 + e^-z) of a pair; the slope is the first times the second's square.
// Below -87 z counts as -87, where the sigmoid is 2^-125.  The reciprocal is the hardware's
// approximation, a step of 2^-23 off at most, after one Newton step: within 1.02 times half a step.
__device__ __forceinline__ void sigmoid_of(uint64_t z, uint64_t& e, uint64_t& r) {
    float lo, hi, a, b;
    f2_unpack(z, lo, hi);
    asm("min.NaN.f32 %0, %1, 0f42AE0000;" : "=f"(lo) : "f"(-lo));  // 87
    asm("min.NaN.f32 %0, %1, 0f42AE0000;" : "=f"(hi) : "f"(-hi));
    e = contract_exp_x2(f2_pack(lo, hi));
    const uint64_t d = f2_add(e, f2_splat(1.0f));
    f2_unpack(d, lo, hi);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(lo));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(hi));
    const uint64_t r0 = f2_pack(a, b);
    const uint64_t off = f2_fma(f2_pack(-lo, -hi), r0, f2_splat(1.0f));
    r = f2_fma(r0, off, r0);
}

// ---------------------------------------------------------------- 8-bit checkpoints
// What a block's byte multiplies its codes by: 2^(b - 133) or 2^(b - 127), the smallest ones
// subnormal, and infinity for 255, whose codes are 0, so that the features come out as NaN.  Codes
// have at most 7 bits, so every product is exact, and a bf16 number unless it is no multiple of 2^-133
// (some e4m3 codes under the bytes 0 to 2, which the quantiser does not write).
template <int kSaved>
__device__ __forceinline__ float saved_scale(uint32_t b) {
    const float s = __uint_as_float(max(b << 23, 0x00400000u));
    return kSaved == RLK_SAVED_INT8 ? __fmul_rn(s, 0x1p-6f) : s;
}

// 8 codes times their block's scale, as 4 packed pairs.
template <int kSaved>
__device__ __forceinline__ void saved_decode8(uint2 codes, float scale, uint64_t (&v)[4]) {
    const uint32_t w[2] = {codes.x, codes.y};
    const uint64_t by = f2_splat(scale);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if (kSaved == RLK_SAVED_INT8) {
            // 2^23 + (code + 128) as a float, less 2^23 + 128
            const uint32_t u = w[p >> 1] ^ 0x80808080u;
            const float lo = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + 2 * (p & 1)));
            const float hi = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + 2 * (p & 1)));
            v[p] = f2_mul(f2_add(f2_pack(lo, hi), f2_splat(-8388736.0f)), by);
        } else {
            // sign, exponent and mantissa in fp32's places: the number times 2^-120, subnormal ones
            // included
            const uint32_t lo = __byte_perm(w[p >> 1], 0u, 0x0444 + 0x2000 * (p & 1));
            const uint32_t hi = __byte_perm(w[p >> 1], 0u, 0x1444 + 0x2000 * (p & 1));
            const uint64_t c = f2_pack(
                __uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(lo) >> 4) & 0x87F00000u),
                __uint_as_float(static_cast<uint32_t>(static_cast<int32_t>(hi) >> 4) & 0x87F00000u));
            v[p] = f2_mul(f2_mul(c, f2_splat(0x1p120f)), by);
        }
    }
}

// The largest magnitude of 8 bf16 numbers, as its bits; NaN counts as the largest of all.
__device__ __forceinline__ uint32_t amax8(uint4 w) {
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16);
}

// The byte of a block whose largest magnitude has these bits.
template <int kSaved>
__device__ __forceinline__ uint32_t saved_byte(uint32_t amax) {
    const int e = static_cast<int>(amax >> 7);
    if (e == 255 || kSaved == RLK_SAVED_INT8) return static_cast<uint32_t>(e);
    const int b = e - 8 + ((amax & 0x7Fu) > 96u && e < 254 ? 1 : 0);
    return static_cast<uint32_t>(b > 0 ? b : 0);
}

// 8 bf16 numbers of a block with this largest magnitude and byte, as codes.  Called by whole warps.
template <int kSaved>
__device__ __forceinline__ uint2 saved_encode8(uint4 x, uint32_t amax, uint32_t b) {
    uint64_t v[4];
    pairs_of(x, v);
    uint32_t q[2];
    if (kSaved == RLK_SAVED_INT8) {
        // the code in the low bits of 1.5 * 2^23 + code, rounded to it by the addition
        float w[8];
        // a block that may hold 127.5 steps, which would be 128, one whose 1 / scale is beyond fp32,
        // or one that is not finite: seldom, and then the warp takes care of all of them
        const bool special = b < 6 || (amax & 0x7Fu) == 0x7Fu || b == 255;
        if (__any_sync(0xffffffffu, special)) {
            const int up = 133 - static_cast<int>(b), first = up < 127 ? up : 127;
            const uint64_t by = f2_splat(__int_as_float((first + 127) << 23));
            const uint64_t more = f2_splat(__int_as_float((up - first + 127) << 23));
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                f2_unpack(f2_fma(f2_mul(v[p], more), by, f2_splat(0x1.8p+23f)), w[2 * p], w[2 * p + 1]);
#pragma unroll
                for (int k = 2 * p; k < 2 * p + 2; ++k)
                    w[k] = b == 255 ? 0.0f : fminf(fmaxf(w[k], 0x1.8p+23f - 127.0f), 0x1.8p+23f + 127.0f);
            }
        } else {
            const uint64_t by = f2_splat(__uint_as_float((260u - b) << 23));
#pragma unroll
            for (int p = 0; p < 4; ++p) f2_unpack(f2_fma(v[p], by, f2_splat(0x1.8p+23f)), w[2 * p], w[2 * p + 1]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            q[k] = __byte_perm(__byte_perm(__float_as_uint(w[4 * k]), __float_as_uint(w[4 * k + 1]), 0x0040),
                               __byte_perm(__float_as_uint(w[4 * k + 2]), __float_as_uint(w[4 * k + 3]), 0x0040), 0x5410);
    } else {
        const uint64_t by = f2_splat(__uint_as_float((254u - b) << 23));
        uint32_t two[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            float lo, hi;
            f2_unpack(f2_mul(v[p], by), lo, hi);
            two[p] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
        }
        q[0] = b == 255 ? 0u : __byte_perm(two[0], two[1], 0x5410);
        q[1] = b == 255 ? 0u : __byte_perm(two[2], two[3], 0x5410);
    }
    return make_uint2(q[0], q[1]);
}

// ---------------------------------------------------------------- sums over a row
// A team of kWarps warps (a power of two) adds up to three sums at once, and each of its threads
// gets them.  The warp's part: `x` and `b` hold a lane's sums of column groups 0 and 1, `d` a single
// one.  Each level halves the lanes that work on a sum while there is another to take the other half,
// so three trees cost little more shuffles than one.  Every tree has the contract's shape: lanes
// 1, 2, .. 16 apart, then the two groups, then the warps pairwise; the sum of two does not depend on
// which is left.  Afterwards lane 0 has x's sum, lane 2 b's, lane 4 d's.
template <bool kThree>
__device__ __forceinline__ float warp_sums(const float (&x)[2], const float (&b)[2], float d) {
    const int lane = threadIdx.x & 31;
    const bool one = lane & 1, two = lane & 2, four = lane & 4;
    const auto far = [](float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); };
    float v = __fadd_rn(one ? x[1] : x[0], far(one ? x[0] : x[1], 1));
    if (kThree) {
        const float w = __fadd_rn(one ? b[1] : b[0], far(one ? b[0] : b[1], 1));
        v = __fadd_rn(two ? w : v, far(two ? v : w, 2));
    } else {
        v = __fadd_rn(v, far(v, 2));
    }
    d = __fadd_rn(d, far(d, 1));
    d = __fadd_rn(d, far(d, 2));
    v = __fadd_rn(four ? d : v, far(four ? v : d, 4));
    v = __fadd_rn(v, far(v, 8));
    v = __fadd_rn(v, far(v, 16));
    const float w = __fadd_rn(v, far(v, 1));  // every lane shuffles
    return four ? v : w;
}

// The warps' parts of a team, kept as rows of four floats: this lane's one of them, added over the
// warps.  Sum `which` ends up in lane which * kWarps (of 16 warps sums 0 and 1 alone, at lanes 0 and 16).
template <int kWarps>
__device__ __forceinline__ float team_sums(const float4* part) {
    const int lane = threadIdx.x & 31;
    float v = reinterpret_cast<const float*>(part + (lane & (kWarps - 1)))[(lane / kWarps) & 3];
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// One of the sums alone, in every lane.
template <int kWarps>
__device__ __forceinline__ float team_sum(const float4* part, int which) {
    float v = reinterpret_cast<const float*>(part + (threadIdx.x & (kWarps - 1)))[which];
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <int kWarps>
__device__ __forceinline__ void team_barrier(int team) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kWarps) : "memory");
}

}  // namespace rlk
