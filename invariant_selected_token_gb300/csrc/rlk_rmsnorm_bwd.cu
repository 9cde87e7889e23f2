// Backward of the strict RMSNorm.  Per row, with x the row that was
// normalised (after the residual addition), dy = grad_out and the forward's
// rstd (the same tree over the same squares, so the same bits):
//
//   up_i   = dy_i gamma_i
//   c      = rstd^2 / H * sum_i up_i x_i
//   grad_x = rstd (up_i - x_i c) + grad_residual_i
//   grad_gamma_i = sum over rows of dy_i x_i rstd
//
// A row's grad_x does not depend on the batch around it.  grad_gamma is
// summed over at most 152 ranges of consecutive rows, one CTA each, in chains
// of 64 rows a team, then over the ranges by a second launch, in an order that
// T, H and the types fix.  Up
// to kRmsBwdClusterRows rows one cluster of 8 CTAs does both in one launch.
//
// Element i = 256 g + 8 l + j is lane l's j-th value of column group g, as in
// the forward; a thread holds 16 features (two groups), so that the shuffles,
// the barrier and the scalar arithmetic of a row are spread over twice as many
// features as with 8.
//
// What bounds it: HBM.  8191 x 8192 in bf16 with residual: 537 MB in 82 us,
// 6.55 TB/s, 0.98 of a plain copy; 4096 x 4096 from fp32 into bf16 with
// residual: 168 MB in 31 us, 0.80 (at 16384 rows 0.94: the rest is the start,
// the tail and the second launch); 64 rows: 5.0 us, latency.  On the way the
// first two took 162 and 66 us with one row at a time, 111 and 37 with the
// next row in registers, 88 and 38 with 16 features a thread and the ring, the
// second 34 with each lane pair copying its own fp32 sectors.
#include <atomic>
#include <cooperative_groups.h>
#include <cstdint>

#include "rlk_contract.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train.cuh"

namespace rlk {
namespace {

namespace cg = cooperative_groups;

// 16-byte pieces of 8 features
template <int kType>
constexpr int kPieces = kType == RLK_DTYPE_F32 ? 2 : 1;

// Threads of a CTA, one CTA per SM.  With 16 warps of up to 128 registers a row's inputs stay in
// registers while its sums go round, but where a row takes all 16: 8192 x 1024 in bf16 15.2 against
// 16.1 us for reading them twice, 8191 x 8192 83.7 against 81.9; with 24 warps they would spill.
constexpr int kThreads = 512;
template <int kWarps>
constexpr bool kKeep = kWarps < 16;

// A team's sums for grad_gamma move from registers to shared memory, 64 bytes a thread, every so
// many rows: additions one after the other round alike where the rows are alike, and drift (2000
// equal rows a team: 494 half-steps off, 25 so).
constexpr int kChain = 64;
constexpr size_t kHeldBytes = size_t(kThreads) * 16 * sizeof(float);

// Stages of a thread's ring: as many, at most 4, as fit into 227 KB.
template <int kGo, int kGx>
constexpr int kRoomFor = (232448 - int(kHeldBytes) - 256) / (kThreads * 32 * (1 + kPieces<kGo> + kPieces<kGx>));
template <int kGo, int kGx>
constexpr int kStages = kRoomFor<kGo, kGx> < 4 ? kRoomFor<kGo, kGx> : 4;

template <int kType>
__device__ __forceinline__ void store8(void* base, int64_t i, const uint64_t (&v)[4]) {
    float e[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) f2_unpack(v[k], e[2 * k], e[2 * k + 1]);
    if constexpr (kType == RLK_DTYPE_F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = make_float4(e[0], e[1], e[2], e[3]);
        p[1] = make_float4(e[4], e[5], e[6], e[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(e[2 * k], e[2 * k + 1]);
            w[k] = static_cast<uint32_t>(__bfloat16_as_ushort(b.x)) |
                   (static_cast<uint32_t>(__bfloat16_as_ushort(b.y)) << 16);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ void copy16(uint4* dst, const char* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_addr(dst)), "l"(src) : "memory");
}

// Features (2p, 2p + 1) of 8 as they lie in memory.
template <int kType>
__device__ __forceinline__ uint64_t pair_at(const uint4 (&w)[kPieces<kType>], int p) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(w);
    if constexpr (kType == RLK_DTYPE_F32)
        return f2_pack(__uint_as_float(q[2 * p]), __uint_as_float(q[2 * p + 1]));
    else
        return f2_pack(__uint_as_float(q[p] << 16), __uint_as_float(q[p] & 0xFFFF0000u));
}

// fp32 features lie 32 bytes a lane.  A warp copies them as they lie in memory, 512 bytes an
// instruction, into two pieces of its own, 64 vectors in a row, of which every other 8 have their
// neighbours exchanged: so the 8 lanes that a shared-memory access serves at a time find one half
// of their features in 8 different places.
__device__ __forceinline__ int f32_place(int vec) { return vec ^ ((vec >> 3) & 1); }
__device__ __forceinline__ void read_f32(uint4 (&w)[2], const uint4* own) {
    const int at = f32_place(2 * (threadIdx.x & 31));
    w[0] = own[at];
    w[1] = own[at ^ 1];
}

// A team of kWarps warps (a power of two) takes a row, a CTA's teams every kTeams-th row of its
// range.  A warp copies its own features of the next kStages rows into its own part of a ring of
// shared memory: the copies need no CTA-wide barrier, and they fly while the current row is
// reduced.  The arithmetic runs two features per instruction, each lane of which rounds
// like the scalar one.  kChained: a team may have more than one chain of rows (65536 x 8192 in bf16
// 572 against 561 us without; instances of their own, since the same code for fewer rows took
// 15.5 instead of 15.2 us at 8192 x 1024).
template <int kWarps, int kGo, int kGx, bool kChained>
__global__ void __launch_bounds__(kThreads, 1) k_rmsnorm_backward(const RmsBwdArgs a) {
    constexpr int kTeams = kThreads / 32 / kWarps, kN = kStages<kGo, kGx>;
    constexpr int kGroup = 1 + kPieces<kGo> + kPieces<kGx>;  // pieces of 8 features
    static_assert(kN >= 2, "a row flies while another is worked on");
    static_assert(kWarps == 1 || kTeams <= 15, "a named barrier (1 .. 15) per team");
    extern __shared__ uint4 ring[];  // [stage][group][piece][thread]: x, grad_out, grad_residual
    __shared__ __align__(16) float2 part[2][kThreads / 32];
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
    auto piece = [&](int stage, int g, int k) { return ring + ((stage * 2 + g) * kGroup + k) * kThreads; };
    // features i .. i + 7, this lane's own, of a bf16 tensor into piece k
    auto copy_bf16 = [&](const void* base, int64_t i, int stage, int g, int k) {
        copy16(piece(stage, g, k) + threadIdx.x, static_cast<const char*>(base) + i * 2);
    };
    // this lane's share of the 256 features of an fp32 one into pieces k, k + 1; H ends at multiples
    // of 64
    auto copy_f32 = [&](const void* base, int64_t i, int stage, int g, int k) {
        uint4* const to = piece(stage, g, k) + (threadIdx.x >> 5) * 64 + f32_place(lane);
        const char* const from = static_cast<const char*>(base) + (i - 4 * lane) * 4;
        const int left = a.H - 512 * warp - 256 * g - 4 * lane;
        if (left > 0) copy16(to, from);
        if (left > 128) copy16(to + 32, from + 512);
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < r1) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t i = t * a.H + i0 + 256 * g;
                if (in[g]) {
                    copy_bf16(a.x, i, stage, g, 0);
                    if (kGo == RLK_DTYPE_BF16) copy_bf16(a.grad_out, i, stage, g, 1);
                    if (kGx == RLK_DTYPE_BF16 && a.grad_res) copy_bf16(a.grad_res, i, stage, g, 1 + kPieces<kGo>);
                }
                if (kGo == RLK_DTYPE_F32) copy_f32(a.grad_out, i, stage, g, 1);
                if (kGx == RLK_DTYPE_F32 && a.grad_res) copy_f32(a.grad_res, i, stage, g, 1 + kPieces<kGo>);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint4 gam[2][1] = {};
#pragma unroll
    for (int g = 0; g < 2; ++g)
        if (in[g]) gam[g][0] = *reinterpret_cast<const uint4*>(a.gamma + i0 + 256 * g);
    uint64_t dg[2][4] = {};
    ulonglong2* const held = reinterpret_cast<ulonglong2*>(ring + kN * 2 * kGroup * kThreads) + threadIdx.x;
    auto add_held = [&] {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const ulonglong2 v = held[k * kThreads];
            dg[k >> 1][2 * (k & 1)] = f2_add(v.x, dg[k >> 1][2 * (k & 1)]);
            dg[k >> 1][2 * (k & 1) + 1] = f2_add(v.y, dg[k >> 1][2 * (k & 1) + 1]);
        }
    };
    auto move_to_held = [&] {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            held[k * kThreads] = make_ulonglong2(dg[k >> 1][2 * (k & 1)], dg[k >> 1][2 * (k & 1) + 1]);
            dg[k >> 1][2 * (k & 1)] = dg[k >> 1][2 * (k & 1) + 1] = 0;
        }
    };
    if (kChained) move_to_held();  // zeros
    int64_t t = r0 + team, chain_end = t + kChain * kTeams;
#pragma unroll
    for (int k = 0; k < kN; ++k) fetch(t + k * kTeams, k);
    int slot = 0, stage = 0;
    for (; t < r1; t += kTeams) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kN - 1) : "memory");
        __syncwarp();
        // the forward's tree over the squares: pairs of features, then lanes, groups and warps
        float s[2];
        uint64_t dot = 0;
        uint4 row_x[2][1] = {}, row_dy[2][kPieces<kGo>] = {};
        auto read = [&](int g) {
            if (!in[g]) return;
            row_x[g][0] = piece(stage, g, 0)[threadIdx.x];
            if constexpr (kGo == RLK_DTYPE_F32) read_f32(row_dy[g], piece(stage, g, 1) + (threadIdx.x >> 5) * 64);
            else row_dy[g][0] = piece(stage, g, 1)[threadIdx.x];
        };
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            read(g);
            const uint4(&x)[1] = row_x[g];
            const uint4(&dy)[kPieces<kGo>] = row_dy[g];
            float s2[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint64_t v = pair_at<RLK_DTYPE_BF16>(x, p);
                float lo, hi;
                f2_unpack(f2_mul(v, v), lo, hi);
                s2[p] = __fadd_rn(lo, hi);
                dot = f2_fma(f2_mul(pair_at<kGo>(dy, p), pair_at<RLK_DTYPE_BF16>(gam[g], p)), v, dot);
            }
            s[g] = __fadd_rn(__fadd_rn(s2[0], s2[1]), __fadd_rn(s2[2], s2[3]));
        }
        float d0, d1;
        f2_unpack(dot, d0, d1);
        float d = __fadd_rn(d0, d1);
        // even lanes go on with the first group, odd ones with the second
        float q = __fadd_rn(odd ? s[1] : s[0], __shfl_xor_sync(0xffffffffu, odd ? s[0] : s[1], 1));
        d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, 1));
#pragma unroll
        for (int o = 2; o < 32; o <<= 1) {
            q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, o));
            d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, o));
        }
        q = __fadd_rn(q, __shfl_xor_sync(0xffffffffu, q, 1));
        if constexpr (kWarps > 1) {
            if (lane == 0) part[slot][team * kWarps + warp] = make_float2(q, d);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kWarps) : "memory");
            float2 p[kWarps];
#pragma unroll
            for (int i = 0; i < kWarps / 2; ++i) {
                const float4 two = reinterpret_cast<const float4*>(&part[slot][team * kWarps])[i];
                p[2 * i] = make_float2(two.x, two.y);
                p[2 * i + 1] = make_float2(two.z, two.w);
            }
#pragma unroll
            for (int n = kWarps / 2; n >= 1; n >>= 1) {
#pragma unroll
                for (int i = 0; i < n; ++i)
                    p[i] = make_float2(__fadd_rn(p[2 * i].x, p[2 * i + 1].x), __fadd_rn(p[2 * i].y, p[2 * i + 1].y));
            }
            q = p[0].x;
            d = p[0].y;
            slot ^= 1;  // a team's warps are never more than one row apart
        }
        // a product with 1 / H is the quotient itself where H is a power of two
        const float mean = pow2 ? __fmul_rn(q, inv_h) : __fdiv_rn(q, h);
        const float rstd = contract_rsqrt(__fadd_rn(mean, a.eps));
        const float c = __fmul_rn(__fmul_rn(rstd, rstd), __fmul_rn(d, inv_h));
        const uint64_t rstd2 = f2_splat(rstd), neg_c2 = f2_splat(-c);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if constexpr (!kKeep<kWarps>) read(g);
            const uint4(&x)[1] = row_x[g];
            const uint4(&dy)[kPieces<kGo>] = row_dy[g];
            uint4 res[kPieces<kGx>] = {};
            if (in[g] && a.grad_res) {
                if constexpr (kGx == RLK_DTYPE_F32) read_f32(res, piece(stage, g, 1 + kPieces<kGo>) + (threadIdx.x >> 5) * 64);
                else res[0] = piece(stage, g, 1 + kPieces<kGo>)[threadIdx.x];
            }
            uint64_t o[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint64_t v = pair_at<RLK_DTYPE_BF16>(x, p), y = pair_at<kGo>(dy, p);
                const uint64_t up = f2_mul(y, pair_at<RLK_DTYPE_BF16>(gam[g], p));
                o[p] = f2_fma(rstd2, f2_fma(v, neg_c2, up), pair_at<kGx>(res, p));
                dg[g][p] = f2_fma(y, f2_mul(v, rstd2), dg[g][p]);
            }
            const int64_t at = t * a.H + i0 + 256 * g;
            if constexpr (kGx == RLK_DTYPE_F32) {
                // even lanes hand their last four features over for the odd ones' first four
                const uint64_t r0 = __shfl_xor_sync(0xffffffffu, odd ? o[0] : o[2], 1);
                const uint64_t r1 = __shfl_xor_sync(0xffffffffu, odd ? o[1] : o[3], 1);
                o[0] = odd ? r0 : o[0];
                o[1] = odd ? r1 : o[1];
                o[2] = odd ? o[2] : r0;
                o[3] = odd ? o[3] : r1;
                float e[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) f2_unpack(o[k], e[2 * k], e[2 * k + 1]);
                if (in[g]) {
                    float* const to = static_cast<float*>(a.grad_x) + at - 4 * odd;
                    *reinterpret_cast<float4*>(to) = make_float4(e[0], e[1], e[2], e[3]);
                    *reinterpret_cast<float4*>(to + 8) = make_float4(e[4], e[5], e[6], e[7]);
                }
            } else if (in[g]) {
                store8<kGx>(a.grad_x, at, o);
            }
        }
        __syncwarp();
        fetch(t + kN * kTeams, stage);  // everything in this stage has been used
        stage = stage + 1 < kN ? stage + 1 : 0;
        if (kChained && t + kTeams == chain_end) {
            add_held();
            move_to_held();
            chain_end += kChain * kTeams;
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!a.grad_gamma) return;
    if (kChained) add_held();
    // the range's sums: the teams' in ascending order.  The ring holds them, once every warp has
    // read its last row out of it.
    float* const teams = reinterpret_cast<float*>(ring);
    float* const sums = teams + kThreads * 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = static_cast<int>(cluster.num_blocks());
    float* const out = ctas > 1 ? sums : a.parts + static_cast<int64_t>(blockIdx.x) * a.H;
    if constexpr (kTeams == 1) {
        if (ctas > 1) __syncthreads();  // `out` lies over other warps' pieces
#pragma unroll
        for (int g = 0; g < 2; ++g)
            if (in[g]) store8<RLK_DTYPE_F32>(out, i0 + 256 * g, dg[g]);
    } else {
        __syncthreads();
#pragma unroll
        for (int g = 0; g < 2; ++g) store8<RLK_DTYPE_F32>(teams, team * kWarps * 512 + i0 + 256 * g, dg[g]);
        __syncthreads();
        for (int i = threadIdx.x; i < a.H; i += kThreads) {
            float v = teams[i];
#pragma unroll
            for (int k = 1; k < kTeams; ++k) v = __fadd_rn(v, teams[k * kWarps * 512 + i]);
            out[i] = v;
        }
    }
    if (ctas > 1) {
        // one cluster: each CTA adds a share of the features over the CTAs, ascending
        cluster.sync();
        for (int i = static_cast<int>(cluster.block_rank()) * kThreads + threadIdx.x; i < a.H; i += ctas * kThreads) {
            float v = cluster.map_shared_rank(sums, 0)[i];
            for (int c = 1; c < ctas; ++c) v = __fadd_rn(v, cluster.map_shared_rank(sums, c)[i]);
            a.grad_gamma[i] = v;
        }
        cluster.sync();  // nobody leaves while its shared memory may be read
    }
}

// grad_gamma from the ranges' sums: 32 threads per feature, each taking every 32nd range in
// ascending order, then pairwise.
__global__ void __launch_bounds__(1024) k_rmsnorm_gamma_sum(const float* parts, int ranges, int H,
                                                            float* out) {
    __shared__ float smem[32][33];
    const int c = threadIdx.x & 31, row = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    ptx::grid_dependency_wait();
    float s = 0.0f;
#pragma unroll 5
    for (int r = row; r < ranges; r += 32) s = __fadd_rn(s, parts[static_cast<int64_t>(r) * H + col]);
    smem[row][c] = s;
    __syncthreads();
    s = warp_sum(smem[c][row]);  // feature `row` of the CTA's 32, one range class per lane
    if (c == 0) out[blockIdx.x * 32 + row] = s;
}

template <int kWarps, int kGo, int kGx, bool kChained>
cudaError_t launch_chained(const RmsBwdArgs& a, int blocks, cudaStream_t stream) {
    constexpr size_t kSmem =
        size_t(kStages<kGo, kGx>) * 2 * (1 + kPieces<kGo> + kPieces<kGx>) * kThreads * sizeof(uint4) +
        (kChained ? kHeldBytes : 0);
    // once per device and kernel: the runtime keeps it, and asking each time costs the host 1 us
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k_rmsnorm_backward<kWarps, kGo, kGx, kChained>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(blocks, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = rmsnorm_backward_one_launch(a.T) && a.grad_gamma ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_rmsnorm_backward<kWarps, kGo, kGx, kChained>, a);
}

template <int kWarps, int kGo, int kGx>
cudaError_t launch_types(const RmsBwdArgs& a, int blocks, cudaStream_t stream) {
    const bool chained = a.grad_gamma && (a.T + int64_t(blocks) - 1) / blocks > kChain * (kThreads / 32 / kWarps);
    return chained ? launch_chained<kWarps, kGo, kGx, true>(a, blocks, stream)
                   : launch_chained<kWarps, kGo, kGx, false>(a, blocks, stream);
}

template <int kWarps>
cudaError_t launch_row(const RmsBwdArgs& a, int blocks, cudaStream_t stream) {
    if (a.go_dtype == RLK_DTYPE_F32)
        return a.gx_dtype == RLK_DTYPE_F32 ? launch_types<kWarps, RLK_DTYPE_F32, RLK_DTYPE_F32>(a, blocks, stream)
                                           : launch_types<kWarps, RLK_DTYPE_F32, RLK_DTYPE_BF16>(a, blocks, stream);
    return a.gx_dtype == RLK_DTYPE_F32 ? launch_types<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_F32>(a, blocks, stream)
                                       : launch_types<kWarps, RLK_DTYPE_BF16, RLK_DTYPE_BF16>(a, blocks, stream);
}

}  // namespace

cudaError_t launch_rmsnorm_backward(const RmsBwdArgs& a, cudaStream_t stream) {
    const bool one = rmsnorm_backward_one_launch(a.T) && a.grad_gamma;
    const int blocks = one ? 8 : rmsnorm_backward_ranges(a.T);
    int warps = 1;
    while (warps * 512 < a.H) warps *= 2;
    cudaError_t e = cudaSuccess;
    if (blocks > 0) switch (warps) {
        case 1: e = launch_row<1>(a, blocks, stream); break;
        case 2: e = launch_row<2>(a, blocks, stream); break;
        case 4: e = launch_row<4>(a, blocks, stream); break;
        case 8: e = launch_row<8>(a, blocks, stream); break;
        case 16: e = launch_row<16>(a, blocks, stream); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || !a.grad_gamma || one) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(a.H / 32, 1, 1);
    cfg.blockDim = dim3(1024, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rmsnorm_gamma_sum, static_cast<const float*>(a.parts), blocks, a.H, a.grad_gamma);
}

}  // namespace rlk
