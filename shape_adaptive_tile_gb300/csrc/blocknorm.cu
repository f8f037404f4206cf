// Block norm (include/rowops.h): checks of arguments, the division of the
// backward pass among CTAs, and the kernel that adds its partial sums.
#include "blocknorm.h"

#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::blocknorm;
using sat::rows::aligned;
using sat::rows::packs;
using sat::rows::type_bytes;
using sat::rows::type_ok;

// The sums of all parts, or of a gate row's pieces, in a fixed order
// (interleaved runs of blockDim.y, then those): a CTA takes 32 columns of one
// sum.
constexpr int kMaxRuns = 32;

struct Outputs {
    float* weights[kSums];  // by Sum; the gate's is not used
    void* dgate;
    int64_t lddg;
    int32_t gate_type;
};

template <typename T>
__device__ __forceinline__ void put(void* p, int64_t at, float v)
{
    static_cast<T*>(p)[at] = rows::from_f32<T>(v);
}

__global__ void __launch_bounds__(32 * kMaxRuns)
    sat_block_norm_sums_kernel(const float* parts, const Split split, int width, const Outputs out)
{
    __shared__ float run[kMaxRuns][32];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // started before the parts were done
    const int c = blockIdx.x * 32 + threadIdx.x;
    // Blocks 0 .. sums - 1 in y: a weight's sum; from there on gate rows.
    const bool gate = blockIdx.y >= split.sums;
    const int sum = gate ? static_cast<int>(kGate) : blockIdx.y;
    if (!gate && (sum == kGate || !out.weights[sum]))
        return;
    const int64_t group = gate ? blockIdx.y - split.sums : 0;
    const int64_t first = gate ? group * split.pieces : 0, end = gate ? first + split.pieces : split.parts;
    float s = 0.0f;
    if (c < width)
        for (int64_t p = first + threadIdx.y; p < end; p += blockDim.y)
            s += parts[(p * split.sums + sum) * split.stride + c];
    run[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= width)
        return;
    for (int l = 1; l < blockDim.y; ++l)
        s += run[l][threadIdx.x];
    if (!gate)
        out.weights[sum][c] = s;
    else if (out.gate_type == GEMM_C_F32)
        put<float>(out.dgate, group * out.lddg + c, s);
    else if (out.gate_type == GEMM_C_BF16)
        put<__nv_bfloat16>(out.dgate, group * out.lddg + c, s);
    else
        put<__half>(out.dgate, group * out.lddg + c, s);
}

Split split_of(const rowop_block_norm_args& a, bool gate)
{
    Split s = {};
    const bool layer = a.post_norm == ROWOP_NORM_LAYER || a.pre_norm == ROWOP_NORM_LAYER;
    s.sums = layer ? kSums : kPreBeta;
    s.mode = !layer ? kRms : a.gate && a.rows_per_gate < a.rows ? kLayerGrouped : kLayerShared;
    s.stride = (a.width + 7) / 8 * 8;
    s.threads = a.width <= 256 ? 32 : a.width <= 1024 ? 128 : a.width <= 2048 ? 256 : 512;
    s.ctas = static_cast<int32_t>((a.width + 4095) / 4096);
    // Parts that run at once: eight warps an SM, CTAs of 512 threads an SM, or
    // as many clusters of these as the GPU's groups of SMs hold (what
    // cudaOccupancyMaxActiveClusters says of a GB300).
    constexpr int64_t clusters[kMaxCluster + 1] = {0, 152, 76, 46, 36};
    const int64_t fill = s.threads == 32 ? kSMs * 8 : clusters[s.ctas] * (512 / s.threads);
    s.group_rows = gate && a.rows_per_gate < a.rows ? a.rows_per_gate : a.rows;
    s.groups = a.rows ? (a.rows + s.group_rows - 1) / s.group_rows : 0;
    if (s.groups > 1 && s.groups >= fill) {
        s.direct = 1;
        s.parts = fill;
    } else if (s.groups) {
        // Pieces of a group: as many as fill the GPU in the fewest rounds of equal parts.
        double best = 1e30;
        for (int64_t rounds = 1; rounds <= 4; ++rounds) {
            int64_t n = rounds * fill / s.groups;
            n = n < 1 ? 1 : n < s.group_rows ? n : s.group_rows;
            const double time = static_cast<double>((s.groups * n + fill - 1) / fill) * ((s.group_rows + n - 1) / n);
            if (time < best * 0.95) {
                best = time;
                s.pieces = n;
            }
        }
        s.parts = s.groups * s.pieces;
        s.direct = s.groups > 1 && s.pieces == 1;
    }
    return s;
}

int check_sizes(const rowop_block_norm_args* a)
{
    if (!a)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    if (a->rows < 0 || a->width < 0)
        return fail_with(GEMM_ERR_ARG, "negative size");
    if (a->rows >= INT64_C(1) << 31)
        return fail_with(GEMM_ERR_ARG, "rows %lld is not below 2^31", (long long)a->rows);
    if (a->width > ROWOP_BLOCK_NORM_MAX_WIDTH)
        return fail_with(GEMM_ERR_ARG, "width %lld is above the %d these kernels hold in registers", (long long)a->width,
                         ROWOP_BLOCK_NORM_MAX_WIDTH);
    if (!type_ok(a->block_type) || (a->stream_type != GEMM_C_F32 && a->stream_type != a->block_type))
        return fail_with(GEMM_ERR_ARG, "bad type: the stream is fp32 or of the block's type");
    if (a->post_norm < ROWOP_NORM_NONE || a->post_norm > ROWOP_NORM_LAYER || a->pre_norm < ROWOP_NORM_NONE ||
        a->pre_norm > ROWOP_NORM_LAYER)
        return fail_with(GEMM_ERR_ARG, "unknown norm");
    if (a->gate && a->gate_type != GEMM_C_F32 && a->gate_type != a->block_type)
        return fail_with(GEMM_ERR_ARG, "bad type: the gate is fp32 or of the block's type");
    if (a->gate && (a->rows_per_gate < 1 || (a->rows_per_gate < a->rows && a->ldg < a->width)))
        return fail_with(GEMM_ERR_ARG, "rows_per_gate below 1, or the gate's row stride below the width");
    return GEMM_OK;
}

// A matrix or vector of the call: missing, misaligned or with too short a stride?
int check_matrix(const char* name, const void* p, int64_t ld, int type, const rowop_block_norm_args* a)
{
    if (!p)
        return fail_with(GEMM_ERR_ARG, "%s is NULL", name);
    if (ld < a->width)
        return fail_with(GEMM_ERR_ARG, "%s: row stride below the width", name);
    if (!aligned(p, type_bytes(type)))
        return fail_with(GEMM_ERR_ALIGN, "%s is not aligned to its elements", name);
    return GEMM_OK;
}

int check_weights(const rowop_block_norm_args* a)
{
    for (const void* p : {static_cast<const void*>(a->post_gamma), static_cast<const void*>(a->post_beta),
                          static_cast<const void*>(a->pre_gamma), static_cast<const void*>(a->pre_beta),
                          static_cast<const void*>(a->post_stats), static_cast<const void*>(a->pre_stats)})
        if (!aligned(p, 4))
            return fail_with(GEMM_ERR_ALIGN, "weights and statistics must be 4-byte aligned");
    if (a->gate && !aligned(a->gate, type_bytes(a->gate_type)))
        return fail_with(GEMM_ERR_ALIGN, "gate is not aligned to its elements");
    return GEMM_OK;
}

bool weights_pack(const rowop_block_norm_args& a)
{
    return a.width % 8 == 0 && packs(a.y, a.ldy, a.block_type) && packs(a.gate, a.rows_per_gate < a.rows ? a.ldg : 0, a.gate_type) &&
           packs(a.post_gamma, 0, GEMM_C_F32) && packs(a.post_beta, 0, GEMM_C_F32) && packs(a.pre_gamma, 0, GEMM_C_F32) &&
           packs(a.pre_beta, 0, GEMM_C_F32);
}

int launched(cudaError_t e)
{
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the block norm: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int rowop_block_norm(const rowop_block_norm_args* args, void* stream)
{
    set_last_error("");
    int rc = check_sizes(args);
    if (rc)
        return rc;
    if (args->rows == 0 || args->width == 0)
        return GEMM_OK;
    const rowop_block_norm_args& a = *args;
    if ((rc = check_matrix("x", a.x, a.ldx, a.stream_type, args)) || (rc = check_matrix("y", a.y, a.ldy, a.block_type, args)) ||
        (rc = check_matrix("h", a.h, a.ldh, a.stream_type, args)) ||
        (a.pre_norm != ROWOP_NORM_NONE && (rc = check_matrix("z", a.z, a.ldz, a.block_type, args))) ||
        (rc = check_weights(args)))
        return rc;
    const bool pack = weights_pack(a) && packs(a.x, a.ldx, a.stream_type) && packs(a.h, a.ldh, a.stream_type) &&
                      (a.pre_norm == ROWOP_NORM_NONE || packs(a.z, a.ldz, a.block_type));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(a.block_type == GEMM_C_F32    ? forward_f32(a, pack, s)
                    : a.block_type == GEMM_C_BF16 ? forward_bf16(a, pack, s)
                                                  : forward_f16(a, pack, s));
}

int64_t rowop_block_norm_workspace(const rowop_block_norm_args* args)
{
    set_last_error("");
    const int rc = check_sizes(args);
    if (rc)
        return rc;
    if (args->rows == 0 || args->width == 0)
        return 0;
    // With the gate's gradient or without: the larger.
    int64_t most = 0;
    for (bool gate : {false, true}) {
        const Split s = split_of(*args, gate && args->gate);
        const int64_t bytes = s.parts * s.sums * s.stride * 4;
        most = bytes > most ? bytes : most;
    }
    return most;
}

int rowop_block_norm_backward(const rowop_block_norm_args* args, const rowop_block_norm_grads* grads, void* stream)
{
    set_last_error("");
    int rc = check_sizes(args);
    if (rc)
        return rc;
    if (!grads)
        return fail_with(GEMM_ERR_ARG, "grads is NULL");
    const rowop_block_norm_args& a = *args;
    const rowop_block_norm_grads& g = *grads;
    const bool pre = a.pre_norm != ROWOP_NORM_NONE, post = a.post_norm != ROWOP_NORM_NONE;
    if ((g.dpre_gamma && !pre) || (g.dpost_gamma && !post) || (g.dpre_beta && a.pre_norm != ROWOP_NORM_LAYER) ||
        (g.dpost_beta && a.post_norm != ROWOP_NORM_LAYER) || (g.dgate && !a.gate))
        return fail_with(GEMM_ERR_ARG, "the gradient of a weight or gate that the call does not have");
    for (const float* p : {g.dpost_gamma, g.dpost_beta, g.dpre_gamma, g.dpre_beta})
        if (!aligned(p, 4))
            return fail_with(GEMM_ERR_ALIGN, "the weights' gradients must be 4-byte aligned");
    if (a.width == 0)
        return GEMM_OK;
    if (a.rows > 0) {
        if ((rc = check_matrix("y", a.y, a.ldy, a.block_type, args)) || (rc = check_weights(args)) ||
            (pre && (rc = check_matrix("h", a.h, a.ldh, a.stream_type, args))) ||
            (pre && (rc = check_matrix("dz", g.dz, g.lddz, a.block_type, args))) ||
            ((!pre || g.dh) && (rc = check_matrix("dh", g.dh, g.lddh, a.stream_type, args))) ||
            (g.dx && (rc = check_matrix("dx", g.dx, g.lddx, a.stream_type, args))) ||
            (g.dy && (rc = check_matrix("dy", g.dy, g.lddy, a.block_type, args))) ||
            (g.dgate && (rc = check_matrix("dgate", g.dgate, a.rows_per_gate < a.rows ? g.lddg : a.width, a.gate_type, args))))
            return rc;
        if ((pre && !a.pre_stats) || (post && !a.post_stats))
            return fail_with(GEMM_ERR_ARG, "the statistics of a norm are NULL");
        if (!g.workspace || g.workspace_bytes < rowop_block_norm_workspace(args))
            return fail_with(GEMM_ERR_ARG, "workspace is NULL or below rowop_block_norm_workspace()");
        if (!aligned(g.workspace, 32))
            return fail_with(GEMM_ERR_ALIGN, "workspace must be 32-byte aligned");
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Split split = split_of(a, g.dgate != nullptr);
    if (a.rows > 0) {
        const bool pack = weights_pack(a) && (!pre || (packs(a.h, a.ldh, a.stream_type) && packs(g.dz, g.lddz, a.block_type))) &&
                          packs(g.dh, g.lddh, a.stream_type) && packs(g.dx, g.lddx, a.stream_type) &&
                          packs(g.dy, g.lddy, a.block_type) && packs(g.dgate, a.rows_per_gate < a.rows ? g.lddg : 0, a.gate_type);
        rc = launched(a.block_type == GEMM_C_F32    ? backward_f32(a, g, split, pack, s)
                      : a.block_type == GEMM_C_BF16 ? backward_bf16(a, g, split, pack, s)
                                                    : backward_f16(a, g, split, pack, s));
        if (rc)
            return rc;
    }
    Outputs out = {};
    out.weights[kPreGamma] = g.dpre_gamma;
    out.weights[kPostGamma] = g.dpost_gamma;
    out.weights[kPreBeta] = g.dpre_beta;
    out.weights[kPostBeta] = g.dpost_beta;
    out.dgate = g.dgate;
    out.lddg = g.lddg;
    out.gate_type = a.gate_type;
    const bool gate_sums = g.dgate && !split.direct;
    if (g.dpre_gamma || g.dpost_gamma || g.dpre_beta || g.dpost_beta || gate_sums) {
        const dim3 grid(static_cast<unsigned>((a.width + 31) / 32),
                        static_cast<unsigned>(split.sums + (gate_sums ? split.groups : 0)));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(32, split.parts > 64 && grid.y <= 16 ? kMaxRuns : 8);  // many gate rows have few pieces each
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        rc = launched(cudaLaunchKernelEx(&cfg, sat_block_norm_sums_kernel, static_cast<const float*>(g.workspace), split,
                                         static_cast<int>(a.width), out));
    }
    return rc;
}

}  // extern "C"
