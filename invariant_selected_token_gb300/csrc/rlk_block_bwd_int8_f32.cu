// The block norms' backward from int8 checkpoints, fp32 grad_out.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_int8_f32(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    return launch_rows<RLK_DTYPE_F32, RLK_SAVED_INT8>(a, blocks, stream);
}

}  // namespace rlk
