// The block norms' backward from e4m3 checkpoints.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_e4m3(const BlockBwdArgs& a, cudaStream_t stream) {
    return launch_block_bwd<RLK_SAVED_E4M3>(a, stream);
}

}  // namespace rlk
