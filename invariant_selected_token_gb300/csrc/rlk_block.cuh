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
// one translation unit for each kind of saved activation
cudaError_t launch_block_bwd_bf16(const BlockBwdArgs& a, cudaStream_t stream);
cudaError_t launch_block_bwd_int8(const BlockBwdArgs& a, cudaStream_t stream);
cudaError_t launch_block_bwd_e4m3(const BlockBwdArgs& a, cudaStream_t stream);

struct VerifyArgs {
    const void* target;          // [rows][ld_target]
    const void* draft;           // [n_draft][ld_draft] or nullptr
    const float* draft_lse;      // [n_draft] or nullptr
    const int32_t* tokens;       // [n_draft]
    const float* uniforms;       // [n_draft]
    const float* noise;          // [n_seqs][ld_noise]
    const int32_t* offsets;      // [n_seqs + 1]
    const uint8_t* active;       // [n_seqs] or nullptr
    const rlk_partial_t* rows;   // [n_draft + n_seqs]: the rows' (m, s)
    const float* lse;            // [n_draft + n_seqs]
    int64_t ld_target, ld_draft, ld_noise;
    int target_dtype, draft_dtype;
    int n_draft, n_seqs, V;
    int32_t* out_accepted;
    int32_t* out_tokens;
    float* out_logprob;
    int32_t* status;
};
cudaError_t launch_draft_verify(const VerifyArgs& a, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- 8-bit checkpoints
// What a block's byte multiplies its codes by.  Both stay exact: a code has at most 7 bits, the
// product is a bf16 number (a subnormal one near the bottom of the range), and 255 is NaN.
template <int kSaved>
__device__ __forceinline__ float saved_scale(uint32_t b) {
    uint32_t bits;
    if (kSaved == RLK_SAVED_INT8)
        bits = b >= 7 ? (b - 6) << 23 : 1u << (b + 16);      // 2^(b - 133)
    else
        bits = b > 0 ? b << 23 : 0x00400000u;                // 2^(b - 127)
    return __uint_as_float(b == 255 ? 0x7FFFFFFFu : bits);
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

__device__ __forceinline__ uint32_t pack_bf16x2(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) |
           (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
}
__device__ __forceinline__ uint64_t unpack_bf16x2(uint32_t w) {
    return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
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

// 8 bf16 numbers of a block with this byte, as codes.
template <int kSaved>
__device__ __forceinline__ uint2 saved_encode8(uint4 x, uint32_t b) {
    if (b == 255) return make_uint2(0u, 0u);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t q[2] = {0u, 0u};
    // 1 / scale, in two factors where it is beyond fp32 (INT8, b below 6)
    const int up = (kSaved == RLK_SAVED_INT8 ? 133 : 127) - static_cast<int>(b);
    const int first = up < 127 ? up : 127;
    const float by = __int_as_float((first + 127) << 23), more = __int_as_float((up - first + 127) << 23);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float lo = __fmul_rn(__fmul_rn(__uint_as_float(w[p] << 16), by), more);
        const float hi = __fmul_rn(__fmul_rn(__uint_as_float(w[p] & 0xFFFF0000u), by), more);
        uint32_t two;
        if (kSaved == RLK_SAVED_INT8) {
            const int a = max(-127, min(127, __float2int_rn(lo))), c = max(-127, min(127, __float2int_rn(hi)));
            two = (static_cast<uint32_t>(a) & 0xFFu) | ((static_cast<uint32_t>(c) & 0xFFu) << 8);
        } else {
            two = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
        }
        q[p >> 1] |= two << (16 * (p & 1));
    }
    return make_uint2(q[0], q[1]);
}

}  // namespace rlk
