// Block norm, forward kernels for blocks in f32.
#include "blocknorm.cuh"

namespace sat {
namespace blocknorm {

cudaError_t forward_f32(const rowop_block_norm_args& a, bool pack, cudaStream_t s)
{
    return forward<float>(a, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
