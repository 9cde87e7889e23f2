// The block norms' backward from e4m3 checkpoints, bf16 grad_out.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_e4m3_bf16(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    return launch_rows<RLK_DTYPE_BF16, RLK_SAVED_E4M3>(a, blocks, stream);
}

}  // namespace rlk
