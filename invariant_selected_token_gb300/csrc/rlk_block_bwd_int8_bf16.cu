// The block norms' backward from int8 checkpoints, bf16 grad_out.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_int8_bf16(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    return launch_rows<RLK_DTYPE_BF16, RLK_SAVED_INT8>(a, blocks, stream);
}

}  // namespace rlk
