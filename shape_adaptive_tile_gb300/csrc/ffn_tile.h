// What the host gives a launch of the feed-forward operators' tile kernel
// (ffn_tile.cuh), and the table of its variants.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace sat {
namespace ffn {

// What becomes of a tile's accumulators.
constexpr int kStore = 0;  // out = alpha acc
constexpr int kGated = 1;  // out = a(alpha gate) (alpha up), and the pre-activations where wanted
constexpr int kGrad = 2;   // dg = dh up a'(gate), du = dh a(gate)

// Operands: the first gives a tile's accumulator rows (128 a CTA), the second
// its columns.
struct TileArgs {
    int tiles_p, tiles_q;  // tiles along the first and the second operand
    int batch;             // 1, or 2 products of one shape (first operands p[z], second q[z], outputs o[z])
    int num_kb;            // k-blocks of a tile, both segments' together
    int seg_kb;            // k-blocks of the first segment: those from seg_kb on come from p[1] and q[1]
    int tail_steps;        // MMA steps of a segment's last k-block (4: all)
    int kb_per_rank;       // split along k: k-blocks of each CTA of the cluster (num_kb where not split)
    int group;             // tile rows that neighbouring CTAs share
    uint32_t idesc;
    float alpha;
    int activation;
    int out_kind;  // 0 fp32, 1 bf16, 2 fp16
    int add;       // kStore, fp32: add to what is there
    int keep;      // kGated: the pre-activations are wanted
    int rows, cols;  // of one output matrix
    int beside;      // this kernel needs nothing of the one before it in the stream, and may run beside it
    void* out[3];    // kStore: batch 0 and 1; kGated: h, gate, up; kGrad: dg, du
    long long ld[3];
    int tma_out;     // bit i: out[i] is written by bulk tensor stores through o[i],
    int tma_edge;    // boxes that reach past the last column too
    int sf_rows_p, sf_rows_q;  // scale rows (512 bytes) of a row tile, i.e. ceil(K / 128); 0 where unscaled
};

struct TileMaps {
    CUtensorMap p[2], q[2];
    CUtensorMap o[3];  // outputs; kGrad: o[2] reads dh
};

struct ScaleMaps {
    CUtensorMap p[2], q[2];
};

struct Variant {
    int mx, epi, cg, bn, p_mn, q_mn, swap;
    int persistent;
    // Of a tile split along k: the ring's bytes, chunks of a tile, and a chunk's sums of one CTA.
    int ring_bytes, chunks, part_bytes;
    cudaError_t (*launch)(const TileMaps& maps, const ScaleMaps* scales, const TileArgs& args, int grid, int cluster,
                          cudaStream_t stream);
    // How many clusters of this many CTAs (up to 8) the current device holds at once.
    cudaError_t (*fit)(int cluster, int* clusters);
};

// A launch that may begin its set-up (up to wait_for_earlier) while the kernel
// before it in the stream ends. A kernel that needs nothing of the one before it
// can do its work at once, and waits before it ends; the one before it then lets
// it begin (launch_dependents) only once it has waited itself, so that all that
// came earlier is over.
template <class... Args>
cudaError_t launch_early(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t stream,
                         Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The variant, or nullptr (ffn_tiles_*.cu).
const Variant* find_variant(int mx, int epi, int cg, int bn, int p_mn, int q_mn, int swap);

}  // namespace ffn
}  // namespace sat
