// Block norm kernels for blocks in f32.
#include "blocknorm.cuh"

namespace sat {
namespace blocknorm {

cudaError_t forward_f32(const rowop_block_norm_args& a, bool pack, cudaStream_t s) { return forward<float>(a, pack, s); }

cudaError_t backward_f32(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                         cudaStream_t s)
{
    return backward<float>(a, g, split, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
