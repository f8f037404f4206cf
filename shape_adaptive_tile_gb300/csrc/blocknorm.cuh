// Block norm and its gradients (include/rowops.h): the kernels and their
// choice, instantiated for one type of the block in each blocknorm_<type>.cu.
//
// NT threads (of one CTA, or of a cluster of CTAs in the backward pass) take
// a row and hold it in registers from its one read to its one write, PER
// columns each. In rows that start on boundaries of eight elements (kPack) a
// thread's columns are groups of eight and each group moves with one 16- or
// 32-byte instruction; otherwise neighbouring threads hold neighbouring
// columns and move them one by one.
#pragma once

#include "blocknorm.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace sat {
namespace blocknorm {

using namespace rows;

// The thread's share of a row: column of its element e of group i.
template <bool kPack, int NT>
__device__ __forceinline__ int column(int lane, int i, int e)
{
    return kPack ? (i * NT + lane) * 8 + e : (i * 8 + e) * NT + lane;
}

// Group i of a row of `width` elements; columns from `width` on are 0.
template <bool kPack, int NT, typename T>
__device__ __forceinline__ void load_group(float (&v)[8], const T* row, int lane, int i, int width)
{
    if constexpr (kPack) {
        const int c = column<true, NT>(lane, i, 0);
        if (c < width) {
            unpack(load_pack(row + c), v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = 0.0f;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false, NT>(lane, i, e);
            v[e] = c < width ? to_f32(row[c]) : 0.0f;
        }
    }
}

template <bool kPack, int NT, typename T>
__device__ __forceinline__ void store_group(T* row, const float (&v)[8], int lane, int i, int width)
{
    if constexpr (kPack) {
        const int c = column<true, NT>(lane, i, 0);
        if (c < width)
            store_pack(row + c, pack<T>(v));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false, NT>(lane, i, e);
            if (c < width)
                row[c] = from_f32<T>(v[e]);
        }
    }
}

// A vector of weights, or `otherwise` where there is none.
template <bool kPack, int NT>
__device__ __forceinline__ void load_weights(float (&v)[8], const float* w, float otherwise, int lane, int i, int width)
{
    if (w) {
        load_group<kPack, NT>(v, w, lane, i, width);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = otherwise;
    }
}

// The gate's row, in its own type: the block's or fp32 (a branch that all threads take alike).
template <bool kPack, int NT, typename B>
__device__ __forceinline__ void load_gate(float (&v)[8], const void* row, bool f32, int lane, int i, int width)
{
    if (!row) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = 1.0f;
    } else if (f32) {
        load_group<kPack, NT>(v, static_cast<const float*>(row), lane, i, width);
    } else {
        load_group<kPack, NT>(v, static_cast<const B*>(row), lane, i, width);
    }
}

__device__ __forceinline__ const void* gate_row(const rowop_block_norm_args& a, int64_t r, int bytes)
{
    return a.gate ? static_cast<const char*>(a.gate) + (a.rows_per_gate >= a.rows ? 0 : r / a.rows_per_gate) * a.ldg * bytes
                  : nullptr;
}

// ---- forward -----------------------------------------------------------------------

// Mean and reciprocal deviation of a row held as NV groups a thread. The
// variance is summed from the deviations, after the mean: the difference of
// two large sums would lose what rows far from 0 have of it.
template <bool kPack, int NT, int NV>
__device__ __forceinline__ void moments(const float (&v)[NV][8], int width, int kind, float eps, int lane, float* scratch,
                                        int& turn, float& mean, float& r)
{
    const float inv = 1.0f / static_cast<float>(width);
    mean = 0.0f;
    if (kind == ROWOP_NORM_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[0] += v[i][e];
        row_sums<NT>(s, scratch, turn);
        mean = s[0] * inv;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = column<kPack, NT>(lane, i, e) < width ? v[i][e] - mean : 0.0f;
            q[0] = fmaf(d, d, q[0]);
        }
    row_sums<NT>(q, scratch, turn);
    r = 1.0f / sqrtf(q[0] * inv + eps);
}

// v = (v - mean) r gamma + beta
template <bool kPack, int NT>
__device__ __forceinline__ void apply(float (&v)[8], float mean, float r, const float* gamma, const float* beta, int lane,
                                      int i, int width)
{
    float g[8], b[8];
    load_weights<kPack, NT>(g, gamma, 1.0f, lane, i, width);
    load_weights<kPack, NT>(b, beta, 0.0f, lane, i, width);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = fmaf((v[e] - mean) * r, g[e], b[e]);
}

template <typename B, typename S, int NT, int NV, bool kPack>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) sat_block_norm_kernel(const __grid_constant__ rowop_block_norm_args a)
{
    __shared__ float scratch[2 * (NT / 32)];
    int turn = 0;
    constexpr int kRows = NT == 32 ? 4 : 1;  // rows of a CTA: a warp each where a warp holds a row
    const int lane = threadIdx.x % NT, width = static_cast<int>(a.width);
    const bool gate_f32 = a.gate_type == GEMM_C_F32;
    const float* post_beta = a.post_norm == ROWOP_NORM_LAYER ? a.post_beta : nullptr;
    const float* pre_beta = a.pre_norm == ROWOP_NORM_LAYER ? a.pre_beta : nullptr;
    for (int64_t r = blockIdx.x * static_cast<int64_t>(kRows) + threadIdx.x / NT; r < a.rows;
         r += gridDim.x * static_cast<int64_t>(kRows)) {
        const B* y = static_cast<const B*>(a.y) + r * a.ldy;
        const S* x = static_cast<const S*>(a.x) + r * a.ldx;
        float v[NV][8], u[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            load_group<kPack, NT>(v[i], y, lane, i, width);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            load_group<kPack, NT>(u[i], x, lane, i, width);
        float mean, rs;
        if (a.post_norm != ROWOP_NORM_NONE) {
            moments<kPack, NT, NV>(v, width, a.post_norm, a.post_eps, lane, scratch, turn, mean, rs);
            if (a.post_stats && lane == 0)
                a.post_stats[2 * r] = mean, a.post_stats[2 * r + 1] = rs;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                apply<kPack, NT>(v[i], mean, rs, a.post_gamma, post_beta, lane, i, width);
        }
        const void* gate = gate_row(a, r, gate_f32 ? 4 : sizeof(B));
        S* h = static_cast<S*>(a.h) + r * a.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float g[8];
            load_gate<kPack, NT, B>(g, gate, gate_f32, lane, i, width);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[i][e] = column<kPack, NT>(lane, i, e) < width
                              ? fmaf(a.residual_scale, u[i][e], a.branch_scale * (v[i][e] * g[e]))
                              : 0.0f;
            store_group<kPack, NT>(h, v[i], lane, i, width);
        }
        if (a.pre_norm == ROWOP_NORM_NONE)
            continue;
        moments<kPack, NT, NV>(v, width, a.pre_norm, a.pre_eps, lane, scratch, turn, mean, rs);
        if (a.pre_stats && lane == 0)
            a.pre_stats[2 * r] = mean, a.pre_stats[2 * r + 1] = rs;
        B* z = static_cast<B*>(a.z) + r * a.ldz;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            apply<kPack, NT>(v[i], mean, rs, a.pre_gamma, pre_beta, lane, i, width);
            store_group<kPack, NT>(z, v[i], lane, i, width);
        }
    }
}

template <typename B, typename S, int NT, int NV, bool kPack>
cudaError_t launch_forward(const rowop_block_norm_args& a, cudaStream_t s)
{
    const int64_t ctas = NT == 32 ? (a.rows + 3) / 4 : a.rows;
    sat_block_norm_kernel<B, S, NT, NV, kPack>
        <<<static_cast<unsigned>(ctas < (1 << 20) ? ctas : (1 << 20)), NT == 32 ? 128 : NT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename B, typename S, bool kPack>
cudaError_t choose_forward(const rowop_block_norm_args& a, cudaStream_t s)
{
    if (a.width <= 256)
        return launch_forward<B, S, 32, 1, kPack>(a, s);
    if (a.width <= 1024)
        return launch_forward<B, S, 128, 1, kPack>(a, s);
    if (a.width <= 2048)
        return launch_forward<B, S, 256, 1, kPack>(a, s);
    if (a.width <= 4096)
        return launch_forward<B, S, 512, 1, kPack>(a, s);
    if (a.width <= 8192)
        return launch_forward<B, S, 512, 2, kPack>(a, s);
    return launch_forward<B, S, 512, 4, kPack>(a, s);
}

// ---- backward ----------------------------------------------------------------------

// The NT threads of CTA `rank` of a cluster of `ctas` take columns
// [rank NT 8, (rank + 1) NT 8) of a row, eight each, and go through one part's
// rows in order, with the sums over rows of their own columns in registers.
template <typename B, typename S, int NT, bool kPack, bool kBeta>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT)
    sat_block_norm_backward_kernel(const __grid_constant__ rowop_block_norm_args a,
                                   const __grid_constant__ rowop_block_norm_grads g, const Split split)
{
    __shared__ float scratch[2 * 2 * (NT / 32)];
    __shared__ float across[2][2][kMaxCluster];
    int turn = 0, cturn = 0;
    constexpr int kParts = NT == 32 ? 4 : 1;
    const int ctas = split.ctas, rank = blockIdx.x % ctas;
    const int64_t part = static_cast<int64_t>(blockIdx.x / ctas) * kParts + threadIdx.x / NT;
    const int lane = threadIdx.x % NT;
    const int off = rank * NT * 8;
    const int64_t whole = a.width;
    const int width = max(0, static_cast<int>(whole) - off);  // columns from `off` on; the threads' share is NT 8 of them
    const float inv = 1.0f / static_cast<float>(whole);
    if (part >= split.parts)
        return;  // only in the one-warp form, which has no barriers

    // Sums over the row: of the CTA's threads, then of the cluster's CTAs in order of rank.
    auto sums = [&](float(&v)[2]) {
        row_sums<NT>(v, scratch, turn);
        if constexpr (NT == 512) {
            if (ctas > 1) {
                if (threadIdx.x < ctas) {
                    const uint32_t at = map_to_cta(smem_u32(&across[cturn][0][rank]), threadIdx.x);
                    st_cluster_f32(at, v[0]);
                    st_cluster_f32(at + kMaxCluster * 4, v[1]);
                }
                __syncwarp();
                cluster_sync();
                v[0] = v[1] = 0.0f;
                for (int c = 0; c < ctas; ++c)
                    v[0] += across[cturn][0][c], v[1] += across[cturn][1][c];
                cturn ^= 1;
            }
        }
    };

    const bool pre = a.pre_norm != ROWOP_NORM_NONE, post = a.post_norm != ROWOP_NORM_NONE;
    const bool pre_layer = a.pre_norm == ROWOP_NORM_LAYER, post_layer = a.post_norm == ROWOP_NORM_LAYER;
    const bool gate_f32 = a.gate_type == GEMM_C_F32;
    const float* post_beta = post_layer && a.post_beta ? a.post_beta + off : nullptr;
    const float* post_gamma = post && a.post_gamma ? a.post_gamma + off : nullptr;
    const float* pre_gamma = pre && a.pre_gamma ? a.pre_gamma + off : nullptr;
    float acc[kBeta ? kSums : kPreBeta][8] = {};
    if constexpr (NT == 512)
        if (ctas > 1)
            cluster_sync();  // the others have started, and may be written to
    int64_t first, end;
    split.range(part, a.rows, first, end);
    int64_t flush = split.direct ? min((first / a.rows_per_gate + 1) * a.rows_per_gate, end) : end;
    for (int64_t r = first; r < end; ++r) {
        float d[8], t[8], w[8], hh[8], sum[2] = {0.0f, 0.0f};
        if (g.dh) {
            load_group<kPack, NT>(d, static_cast<const S*>(g.dh) + r * g.lddh + off, lane, 0, width);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] = 0.0f;
        }
        if (pre) {
            const float mean = a.pre_stats[2 * r], rs = a.pre_stats[2 * r + 1];
            load_group<kPack, NT>(t, static_cast<const B*>(g.dz) + r * g.lddz + off, lane, 0, width);
            load_group<kPack, NT>(hh, static_cast<const S*>(a.h) + r * a.ldh + off, lane, 0, width);
            load_weights<kPack, NT>(w, pre_gamma, 1.0f, lane, 0, width);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hh[e] = (hh[e] - mean) * rs;  // of a column past the row's end: not 0, but t is
                acc[kPreGamma][e] = fmaf(t[e], hh[e], acc[kPreGamma][e]);
                if constexpr (kBeta)
                    acc[kPreBeta][e] += t[e];
                t[e] *= w[e];
                sum[0] = fmaf(t[e], hh[e], sum[0]);
                sum[1] += t[e];
            }
            sums(sum);
            const float s1 = sum[0] * inv, s0 = pre_layer ? sum[1] * inv : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] += column<kPack, NT>(lane, 0, e) < width ? rs * (t[e] - s0 - hh[e] * s1) : 0.0f;
        }
        if (g.dx) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = a.residual_scale * d[e];
            store_group<kPack, NT>(static_cast<S*>(g.dx) + r * g.lddx + off, t, lane, 0, width);
        }
        const float mean = post ? a.post_stats[2 * r] : 0.0f, rs = post ? a.post_stats[2 * r + 1] : 1.0f;
        load_group<kPack, NT>(hh, static_cast<const B*>(a.y) + r * a.ldy + off, lane, 0, width);
        load_weights<kPack, NT>(w, post_gamma, 1.0f, lane, 0, width);
        load_weights<kPack, NT>(t, post_beta, 0.0f, lane, 0, width);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hh[e] = (hh[e] - mean) * rs;
            d[e] *= a.branch_scale;
            acc[kGate][e] = fmaf(d[e], fmaf(hh[e], w[e], t[e]), acc[kGate][e]);
        }
        const char* gate = static_cast<const char*>(gate_row(a, r, gate_f32 ? 4 : sizeof(B)));
        load_gate<kPack, NT, B>(t, gate ? gate + off * (gate_f32 ? 4 : sizeof(B)) : nullptr, gate_f32, lane, 0, width);
        sum[0] = sum[1] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            d[e] *= t[e];
            acc[kPostGamma][e] = fmaf(d[e], hh[e], acc[kPostGamma][e]);
            if constexpr (kBeta)
                acc[kPostBeta][e] += d[e];
            d[e] *= w[e];
            sum[0] = fmaf(d[e], hh[e], sum[0]);
            sum[1] += d[e];
        }
        if (post) {
            sums(sum);
            const float s1 = sum[0] * inv, s0 = post_layer ? sum[1] * inv : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                d[e] = rs * (d[e] - s0 - hh[e] * s1);
        }
        if (g.dy)
            store_group<kPack, NT>(static_cast<B*>(g.dy) + r * g.lddy + off, d, lane, 0, width);
        if (split.direct && r + 1 == flush) {  // the gate row's last row
            if (g.dgate) {
                const int64_t at = r / a.rows_per_gate * g.lddg + off;
                if (gate_f32)
                    store_group<kPack, NT>(static_cast<float*>(g.dgate) + at, acc[kGate], lane, 0, width);
                else
                    store_group<kPack, NT>(static_cast<B*>(g.dgate) + at, acc[kGate], lane, 0, width);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[kGate][e] = 0.0f;
            flush = min(flush + a.rows_per_gate, end);
        }
    }
    // A CTA of a cluster must not end while another may still write to its `across`.
    if constexpr (NT == 512)
        if (ctas > 1)
            cluster_sync();
    float* out = static_cast<float*>(g.workspace) + part * split.sums * split.stride + off;
#pragma unroll
    for (int s = 0; s < (kBeta ? kSums : kPreBeta); ++s)
        store_group<kPack, NT>(out + s * split.stride, acc[s], lane, 0, width);
}

template <typename B, typename S, int NT, bool kPack, bool kBeta>
cudaError_t launch_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(NT == 32 ? (split.parts + 3) / 4 : split.parts * split.ctas));
    cfg.blockDim = dim3(NT == 32 ? 128 : NT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split.ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = NT == 512 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, sat_block_norm_backward_kernel<B, S, NT, kPack, kBeta>, a, g, split);
}

template <typename B, typename S, bool kPack, bool kBeta>
cudaError_t choose_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    switch (backward_threads(a.width)) {
    case 32: return launch_backward<B, S, 32, kPack, kBeta>(a, g, split, s);
    case 128: return launch_backward<B, S, 128, kPack, kBeta>(a, g, split, s);
    case 256: return launch_backward<B, S, 256, kPack, kBeta>(a, g, split, s);
    default: return launch_backward<B, S, 512, kPack, kBeta>(a, g, split, s);
    }
}

// ---- the type of the stream: fp32 or the block's ----------------------------------

template <typename B>
cudaError_t forward(const rowop_block_norm_args& a, bool pack, cudaStream_t s)
{
    if constexpr (!std::is_same_v<B, float>)
        if (a.stream_type == GEMM_C_F32)
            return pack ? choose_forward<B, float, true>(a, s) : choose_forward<B, float, false>(a, s);
    return pack ? choose_forward<B, B, true>(a, s) : choose_forward<B, B, false>(a, s);
}

template <typename B, typename S>
cudaError_t backward_as(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                        cudaStream_t s)
{
    if (split.sums == kSums)
        return pack ? choose_backward<B, S, true, true>(a, g, split, s) : choose_backward<B, S, false, true>(a, g, split, s);
    return pack ? choose_backward<B, S, true, false>(a, g, split, s) : choose_backward<B, S, false, false>(a, g, split, s);
}

template <typename B>
cudaError_t backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split, bool pack,
                     cudaStream_t s)
{
    if constexpr (!std::is_same_v<B, float>)
        if (a.stream_type == GEMM_C_F32)
            return backward_as<B, float>(a, g, split, pack, s);
    return backward_as<B, B>(a, g, split, pack, s);
}

}  // namespace blocknorm
}  // namespace sat
