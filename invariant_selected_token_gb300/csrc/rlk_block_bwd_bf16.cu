// The block norms' backward from bf16 activations.
#include "rlk_block_bwd.cuh"

namespace rlk {

cudaError_t launch_block_bwd_bf16(const BlockBwdArgs& a, cudaStream_t stream) {
    return launch_block_bwd<RLK_SAVED_BF16>(a, stream);
}

}  // namespace rlk
