// Block norm, forward kernels for blocks in f16.
#include "blocknorm.cuh"

namespace sat {
namespace blocknorm {

cudaError_t forward_f16(const rowop_block_norm_args& a, bool pack, cudaStream_t s)
{
    return forward<__half>(a, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
