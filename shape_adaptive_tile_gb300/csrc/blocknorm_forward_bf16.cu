// Block norm, forward kernels for blocks in bf16.
#include "blocknorm.cuh"

namespace sat {
namespace blocknorm {

cudaError_t forward_bf16(const rowop_block_norm_args& a, bool pack, cudaStream_t s)
{
    return forward<__nv_bfloat16>(a, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
