// The block norm's division of rows among CTAs, and its kernels' entries.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "rowops.h"

namespace sat {
namespace blocknorm {

constexpr int64_t kSMs = 152;
constexpr int kSmemPerSM = 227 * 1024;
constexpr int kMaxCluster = 4;  // CTAs that share a row in the backward pass

// The backward pass's parts: each is a range of rows that one warp, CTA or
// cluster goes through, and leaves its sums over. `groups` is the number of
// gate rows whose gradients are wanted (1 without). A part either has whole
// groups (direct: it writes their gate gradients itself) or one of `pieces`
// equal pieces of one group.
struct Split {
    int64_t parts, groups, pieces, group_rows, stride;
    int32_t sums, ctas, direct, threads, mode;

    __host__ __device__ void range(int64_t part, int64_t rows, int64_t& first, int64_t& end) const
    {
        if (direct) {
            first = part * groups / parts * group_rows;
            end = (part + 1) * groups / parts * group_rows;
            end = end < rows ? end : rows;
        } else {
            const int64_t start = part / pieces * group_rows, j = part % pieces;
            const int64_t len = group_rows < rows - start ? group_rows : rows - start;
            first = start + j * len / pieces;
            end = start + (j + 1) * len / pieces;
        }
    }
};

// The sums over rows that a part leaves in the workspace, `stride` floats
// each. Without a Layer norm there are none for betas (sums = kPreBeta).
enum Sum { kPreGamma, kPostGamma, kGate, kPreBeta, kPostBeta, kSums };

// What the backward pass's kernels are compiled for: no Layer norm, or one,
// with a gate that all rows share (or none) or one that changes from row to row.
enum Mode { kRms, kLayerShared, kLayerGrouped };

// CTAs an SM that the backward pass is made for, by their threads: eight
// columns a thread, a warp for rows of up to 256 columns, a cluster for those
// of over 4096.
template <int NT>
constexpr int kBackwardPerSM = 512 / NT;

// Kernels of one block type (blocknorm_<type>.cu). `pack`: all rows start on boundaries of eight elements.
cudaError_t forward_f32(const rowop_block_norm_args& a, bool pack, cudaStream_t s);
cudaError_t forward_bf16(const rowop_block_norm_args& a, bool pack, cudaStream_t s);
cudaError_t forward_f16(const rowop_block_norm_args& a, bool pack, cudaStream_t s);
cudaError_t backward_f32(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                         cudaStream_t s);
cudaError_t backward_bf16(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                          cudaStream_t s);
cudaError_t backward_f16(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                         cudaStream_t s);

}  // namespace blocknorm
}  // namespace sat
