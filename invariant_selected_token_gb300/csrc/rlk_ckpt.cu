// Activation checkpoints in 8 bits: a bf16 tensor to codes with a byte per 32
// features, and back.  Per block of 32 features, with m the largest magnitude,
// the byte is m's exponent (shifted by what the code's own range takes) and a
// code is x / 2^(byte - bias) to the nearest, ties to even.
//
// The tensor is one run of blocks, H being a multiple of 32.  To codes a thread takes
// 16 features, a pair of lanes a block, so that it writes 16 bytes; back it takes
// 8, so that the bf16 that a warp writes at a time lie side by side (16 of them
// in two stores a lane: 34.5 instead of 31.1 us), and two such chunks, a CTA apart, to have
// two reads under way (one: 40, four: 31.8 us).
//
// What bounds it: HBM.  16385 x 4096 takes 30.7 us to codes and 31.2 back, 0.98 of the copy
// rate; 4096 x 4096 9.6 each (0.79), 256 x 4096 1.8, a launch's latency.
#include <cstdint>

#include "rlk_block.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;

template <int kSaved>
__global__ void __launch_bounds__(kThreads)
    k_act_quantize(const uint16_t* x, int64_t chunks, uint8_t* codes, uint8_t* scales) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    const int lane = threadIdx.x & 31;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x - lane; first < chunks; first += stride) {
        const int64_t c = first + lane;
        const bool in = c < chunks;
        uint4 a = {}, b = {};
        if (in) {
            a = reinterpret_cast<const uint4*>(x)[2 * c];
            b = reinterpret_cast<const uint4*>(x)[2 * c + 1];
        }
        uint32_t m = max(amax8(a), amax8(b));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t byte = saved_byte<kSaved>(m);
        const uint2 lo = saved_encode8<kSaved>(a, m, byte), hi = saved_encode8<kSaved>(b, m, byte);
        if (in) reinterpret_cast<uint4*>(codes)[c] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        if (in && !(lane & 1)) scales[c >> 1] = static_cast<uint8_t>(byte);
    }
}

constexpr int kAhead = 2;  // chunks of 8 features that a thread of the restoring kernel has under way

template <int kSaved>
__global__ void __launch_bounds__(kThreads)
    k_act_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t chunks, uint16_t* out) {
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kThreads * kAhead);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kAhead) + threadIdx.x; first < chunks; first += stride) {
        uint2 q[kAhead];
        uint32_t byte[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t c = first + k * kThreads;
            if (c >= chunks) continue;
            q[k] = reinterpret_cast<const uint2*>(codes)[c];
            byte[k] = scales[c >> 2];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t c = first + k * kThreads;
            if (c >= chunks) continue;
            uint64_t v[4];
            saved_decode8<kSaved>(q[k], saved_scale<kSaved>(byte[k]), v);
            reinterpret_cast<uint4*>(out)[c] = words_of(v);
        }
    }
}

// A CTA for each `per` chunks: a launch capped at 32 CTAs an SM, whose CTAs go on with further chunks, takes
// 31.3 instead of 30.7 us (16385 x 4096 to codes).  The cap that is left keeps the grid within its limit.
int blocks_for(int64_t chunks, int64_t per, int num_sms) {
    const int64_t need = (chunks + per - 1) / per, most = static_cast<int64_t>(num_sms) * 1024;
    return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_act_quantize(const uint16_t* x, int format, int64_t n, SavedOut out, int num_sms,
                                cudaStream_t stream) {
    const int64_t chunks = n / 16;
    if (chunks == 0) return cudaSuccess;
    const int blocks = blocks_for(chunks, kThreads, num_sms);
    if (format == RLK_SAVED_INT8)
        k_act_quantize<RLK_SAVED_INT8><<<blocks, kThreads, 0, stream>>>(x, chunks, static_cast<uint8_t*>(out.codes), out.scales);
    else
        k_act_quantize<RLK_SAVED_E4M3><<<blocks, kThreads, 0, stream>>>(x, chunks, static_cast<uint8_t*>(out.codes), out.scales);
    return cudaGetLastError();
}

cudaError_t launch_act_dequantize(SavedIn in, int format, int64_t n, uint16_t* out, int num_sms,
                                  cudaStream_t stream) {
    const int64_t chunks = n / 8;
    if (chunks == 0) return cudaSuccess;
    const int blocks = blocks_for(chunks, kThreads * kAhead, num_sms);
    if (format == RLK_SAVED_INT8)
        k_act_dequantize<RLK_SAVED_INT8><<<blocks, kThreads, 0, stream>>>(static_cast<const uint8_t*>(in.data), in.scales, chunks, out);
    else
        k_act_dequantize<RLK_SAVED_E4M3><<<blocks, kThreads, 0, stream>>>(static_cast<const uint8_t*>(in.data), in.scales, chunks, out);
    return cudaGetLastError();
}

}  // namespace rlk
