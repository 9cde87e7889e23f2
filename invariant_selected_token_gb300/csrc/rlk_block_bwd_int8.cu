// The block norms' backward from int8 checkpoints.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_int8(const BlockBwdArgs& a, cudaStream_t stream) {
    return launch_block_bwd<RLK_SAVED_INT8>(a, stream);
}

}  // namespace rlk
