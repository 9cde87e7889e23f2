// The block norms' backward from e4m3 checkpoints, fp32 grad_out.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_e4m3_f32(const BlockBwdArgs& a, int blocks, cudaStream_t stream) {
    return launch_rows<RLK_DTYPE_F32, RLK_SAVED_E4M3>(a, blocks, stream);
}

}  // namespace rlk
