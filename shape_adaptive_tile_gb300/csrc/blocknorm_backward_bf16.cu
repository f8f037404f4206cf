// Block norm, backward kernels for blocks in bf16.
#include "blocknorm.cuh"

namespace sat {
namespace blocknorm {

cudaError_t backward_bf16(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack, cudaStream_t s)
{
    return backward<__nv_bfloat16>(a, g, split, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
