// Block norm and its gradients (include/rowops.h): the kernels and their
// choice, instantiated for one type of the block in each blocknorm_<type>.cu.
//
// HBM bandwidth bounds both directions: every row is read once and written
// once. NT threads hold a row in registers, eight or more columns each. In
// rows that start on boundaries of eight elements (kPack) a thread's columns
// are groups of eight, moved by one 16- or 32-byte instruction; otherwise
// neighbouring threads hold neighbouring columns and move them one by one.
//
// Where there are more rows than CTAs, a CTA stays for many: a warp of its own
// keeps the next rows on their way into a ring in shared memory (Ring), so
// that memory does not wait for the two reductions that each row has between
// its read and its write.
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

// ---- rows through shared memory ------------------------------------------------------

constexpr int kMaxStages = 8;
constexpr int kWaitLimit = 1 << 22;  // polls of a barrier, each of which the hardware suspends for a while

// One of the matrices that a kernel reads row by row (none where p is NULL).
struct Source {
    const char* p;    // the CTA's first column of row 0
    int64_t pitch;    // bytes from row to row
    int bytes;        // of the CTA's share of a row
    int offset;       // where it lies in a stage

    __device__ __forceinline__ uint64_t row(int64_t r) const { return reinterpret_cast<uint64_t>(p + r * pitch); }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A ring of `stages` stages, each with a row of every source: filled by one
// warp (Ring::fill), read by `warps` others (Ring::take, Ring::release). Bulk
// copies move what lies between 16-byte boundaries of memory; where rows do
// not start on them (not kPack), a row lies in its stage as many bytes after
// a boundary as in memory, and the warp moves its ends by plain loads.
struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];

    __device__ __forceinline__ void init(int stages, int warps)
    {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), warps);
        }
        fence_mbar_init();
    }

    static __device__ __forceinline__ void wait(uint64_t* bar, int parity, bool& failed)
    {
        for (int n = 0; !failed && !mbar_try_wait<true>(smem_u32(bar), parity); ++n)
            failed = n > kWaitLimit;
    }

    template <bool kPack, int N>
    __device__ __forceinline__ void fill(unsigned char* stage, int s, int round, const Source (&sources)[N], int64_t r,
                                         bool& failed)
    {
        const int lane = threadIdx.x % 32;
        wait(&empty[s], round & 1 ^ 1, failed);
        uint32_t total = 0;
        if constexpr (kPack) {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (sources[i].p && sources[i].bytes > 0)
                        total += sources[i].bytes;
                mbar_arrive_expect_tx(smem_u32(&full[s]), total);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (sources[i].p && sources[i].bytes > 0)
                        bulk_load(smem_u32(stage) + sources[i].offset, sources[i].row(r), sources[i].bytes, smem_u32(&full[s]));
            }
            __syncwarp();
        } else {
            fence_proxy_async_smem();  // of the ends written here before
            __syncwarp();
            uint16_t ends[N];
            // The ends in pieces of two bytes: the first eight lanes before the first boundary, the next after the last.
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t lo = sources[i].row(r), hi = lo + sources[i].bytes, lo16 = (lo + 15) & ~15ull, hi16 = hi & ~15ull;
                if (!sources[i].p || sources[i].bytes <= 0)
                    continue;
                const uint32_t bytes = lo16 < hi16 ? static_cast<uint32_t>(hi16 - lo16) : 0;
                total += bytes;
                if (lane == 0 && bytes)
                    bulk_load(smem_u32(stage) + sources[i].offset + static_cast<uint32_t>(lo16 - (lo & ~15ull)), lo16, bytes,
                              smem_u32(&full[s]));
                const uint64_t x = (lane < 8 ? lo & ~15ull : hi16) + lane % 8 * 2;
                if (lane < 16 && x >= lo && x < hi && (x < lo16 || x >= hi16) && (lane < 8 || hi16 >= lo16))
                    ends[i] = *reinterpret_cast<const uint16_t*>(x);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t lo = sources[i].row(r), hi = lo + sources[i].bytes, lo16 = (lo + 15) & ~15ull, hi16 = hi & ~15ull;
                if (!sources[i].p || sources[i].bytes <= 0)
                    continue;
                const uint64_t x = (lane < 8 ? lo & ~15ull : hi16) + lane % 8 * 2;
                if (lane < 16 && x >= lo && x < hi && (x < lo16 || x >= hi16) && (lane < 8 || hi16 >= lo16))
                    *reinterpret_cast<uint16_t*>(stage + sources[i].offset + (x - (lo & ~15ull))) = ends[i];
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(smem_u32(&full[s]), total);
        }
    }

    __device__ __forceinline__ void take(int s, int round, bool& failed) { wait(&full[s], round & 1, failed); }

    __device__ __forceinline__ void release(int s)
    {
        __syncwarp();
        if (threadIdx.x % 32 == 0)
            mbar_arrive(smem_u32(&empty[s]));
    }
};

// Group i of a row of `width` elements that lies in a stage; columns from `width` on are 0.
template <bool kPack, int NT, typename T>
__device__ __forceinline__ void stage_group(float (&v)[8], const unsigned char* stage, const Source& source, int64_t r, int lane,
                                            int i, int width)
{
    if constexpr (kPack) {
        const int c = column<true, NT>(lane, i, 0);
        if (c < width) {
            const uint4* at = reinterpret_cast<const uint4*>(stage + source.offset + c * sizeof(T));
            if constexpr (sizeof(T) == 4) {
                const uint4 a = at[0], b = at[1];
                unpack(Pack<T>{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}, v);
            } else {
                const uint4 a = at[0];
                unpack(Pack<T>{{a.x, a.y, a.z, a.w}}, v);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = 0.0f;
        }
    } else {
        const T* at = reinterpret_cast<const T*>(stage + source.offset + (source.row(r) & 15));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false, NT>(lane, i, e);
            v[e] = c < width ? to_f32(at[c]) : 0.0f;
        }
    }
}

// Sums of N values over the NT threads that come before the filling warp, as
// row_sums, behind a barrier of theirs alone.
template <int NT, int N>
__device__ __forceinline__ void ring_sums(float (&v)[N], float* scratch, int& turn)
{
    constexpr int W = NT / 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* half = scratch + turn * (N * W);
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            half[i * W + warp] = v[i];
    named_bar_sync(1, NT);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = half[i * W + lane % W];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// ---- forward -----------------------------------------------------------------------

// Mean and reciprocal deviation of a row held as NV groups a thread. The
// variance is summed from the deviations, after the mean: the difference of
// two large sums would lose what rows far from 0 have of it.
template <bool kPack, int NT, int NV, typename Sums>
__device__ __forceinline__ void moments(const float (&v)[NV][8], int width, int kind, float eps, int lane, Sums sums,
                                        float& mean, float& r)
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
        sums(s);
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
    sums(q);
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

// What follows a row's read: v is y's share, x(i) gives x's groups; writes h,
// z and the statistics. `lane` is the thread's place among the NT of its row.
template <typename B, typename S, int NT, int NV, bool kPack, typename X, typename Sums>
__device__ __forceinline__ void finish_row(const rowop_block_norm_args& a, int64_t r, float (&v)[NV][8], int lane, X x, Sums sums)
{
    const int width = static_cast<int>(a.width);
    const bool gate_f32 = a.gate_type == GEMM_C_F32;
    float mean, rs;
    if (a.post_norm != ROWOP_NORM_NONE) {
        moments<kPack, NT, NV>(v, width, a.post_norm, a.post_eps, lane, sums, mean, rs);
        if (a.post_stats && lane == 0)
            a.post_stats[2 * r] = mean, a.post_stats[2 * r + 1] = rs;
        const float* beta = a.post_norm == ROWOP_NORM_LAYER ? a.post_beta : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            apply<kPack, NT>(v[i], mean, rs, a.post_gamma, beta, lane, i, width);
    }
    const void* gate = gate_row(a, r, gate_f32 ? 4 : sizeof(B));
    S* h = static_cast<S*>(a.h) + r * a.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float g[8], u[8];
        x(u, i);
        load_gate<kPack, NT, B>(g, gate, gate_f32, lane, i, width);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = column<kPack, NT>(lane, i, e) < width ? fmaf(a.residual_scale, u[e], a.branch_scale * (v[i][e] * g[e])) : 0.0f;
        store_group<kPack, NT>(h, v[i], lane, i, width);
    }
    if (a.pre_norm == ROWOP_NORM_NONE)
        return;
    moments<kPack, NT, NV>(v, width, a.pre_norm, a.pre_eps, lane, sums, mean, rs);
    if (a.pre_stats && lane == 0)
        a.pre_stats[2 * r] = mean, a.pre_stats[2 * r + 1] = rs;
    const float* beta = a.pre_norm == ROWOP_NORM_LAYER ? a.pre_beta : nullptr;
    B* z = static_cast<B*>(a.z) + r * a.ldz;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        apply<kPack, NT>(v[i], mean, rs, a.pre_gamma, beta, lane, i, width);
        store_group<kPack, NT>(z, v[i], lane, i, width);
    }
}

// Few rows, or narrow ones that a warp holds: rows straight into registers.
template <typename B, typename S, int NT, int NV, bool kPack>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) sat_block_norm_kernel(const __grid_constant__ rowop_block_norm_args a)
{
    __shared__ float scratch[2 * (NT / 32)];
    int turn = 0;
    constexpr int kRows = NT == 32 ? 4 : 1;  // rows of a CTA: a warp each where a warp holds a row
    const int lane = threadIdx.x % NT, width = static_cast<int>(a.width);
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
        finish_row<B, S, NT, NV, kPack>(
            a, r, v, lane,
            [&](float(&to)[8], int i) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    to[e] = u[i][e];
            },
            [&](float(&s)[1]) { row_sums<NT>(s, scratch, turn); });
    }
}

// Many rows: a CTA's NT threads take every gridDim.x-th, through a ring of
// `stages` stages of `stage_bytes`.
template <typename B, typename S, int NT, int NV, bool kPack>
__global__ void __launch_bounds__(NT + 32, NT == 512 ? (NV == 4 ? 1 : 2) : NT == 256 ? 3 : 5)
    sat_block_norm_ring_kernel(const __grid_constant__ rowop_block_norm_args a, int stages, int stage_bytes)
{
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ __align__(8) Ring ring;
    __shared__ float scratch[2 * (NT / 32)];
    const int width = static_cast<int>(a.width);
    const int y_bytes = (width * static_cast<int>(sizeof(B)) + 31) / 16 * 16;
    const Source sources[2] = {
        {static_cast<const char*>(a.y), a.ldy * static_cast<int64_t>(sizeof(B)), width * static_cast<int>(sizeof(B)), 0},
        {static_cast<const char*>(a.x), a.ldx * static_cast<int64_t>(sizeof(S)), width * static_cast<int>(sizeof(S)), y_bytes}};
    if (threadIdx.x == 0)
        ring.init(stages, NT / 32);
    __syncthreads();
    bool failed = false;
    int s = 0, round = 0, turn = 0;
    if (threadIdx.x >= NT) {
        for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
            ring.fill<kPack>(ring_memory + s * stage_bytes, s, round, sources, r, failed);
            if (++s == stages)
                s = 0, ++round;
        }
        return;
    }
    const int lane = threadIdx.x;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        ring.take(s, round, failed);
        const unsigned char* stage = ring_memory + s * stage_bytes;
        float v[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            stage_group<kPack, NT, B>(v[i], stage, sources[0], r, lane, i, width);
            if (failed)
                v[i][0] = NAN;
        }
        finish_row<B, S, NT, NV, kPack>(
            a, r, v, lane,
            [&](float(&to)[8], int i) {
                stage_group<kPack, NT, S>(to, stage, sources[1], r, lane, i, width);
                if (i == NV - 1)
                    ring.release(s);
            },
            [&](float(&v)[1]) { ring_sums<NT>(v, scratch, turn); });
        if (++s == stages)
            s = 0, ++round;
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

template <typename B, typename S, int NT, int NV, bool kPack>
cudaError_t launch_ring(const rowop_block_norm_args& a, cudaStream_t s)
{
    constexpr int per_sm = NT == 512 ? (NV == 4 ? 1 : 2) : NT == 256 ? 3 : 5;
    if (a.rows < 2 * per_sm * kSMs)  // under two rows a CTA there is nothing to fetch ahead
        return launch_forward<B, S, NT, NV, kPack>(a, s);
    const int64_t w = a.width;
    const int stage = static_cast<int>((w * sizeof(B) + 31) / 16 * 16 + (w * sizeof(S) + 31) / 16 * 16);
    const int room = kSmemPerSM / per_sm - 1024;
    int stages = room / stage;
    stages = stages < kMaxStages ? stages : kMaxStages;
    auto kernel = sat_block_norm_ring_kernel<B, S, NT, NV, kPack>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel), room);
    if (e != cudaSuccess)
        return e;
    kernel<<<static_cast<unsigned>(per_sm * kSMs), NT + 32, stages * stage, s>>>(a, stages, stage);
    return cudaGetLastError();
}

template <typename B, typename S, bool kPack>
cudaError_t choose_forward(const rowop_block_norm_args& a, cudaStream_t s)
{
    if (a.width <= 256)
        return launch_forward<B, S, 32, 1, kPack>(a, s);
    if (a.width <= 1024)
        return launch_ring<B, S, 128, 1, kPack>(a, s);
    if (a.width <= 2048)
        return launch_ring<B, S, 256, 1, kPack>(a, s);
    if (a.width <= 4096)
        return launch_ring<B, S, 512, 1, kPack>(a, s);
    if (a.width <= 8192)
        return launch_ring<B, S, 512, 2, kPack>(a, s);
    return launch_ring<B, S, 512, 4, kPack>(a, s);
}

// ---- backward ----------------------------------------------------------------------

// The sources of the backward pass, and its weights.
enum Input { kDh, kDz, kH, kY, kInputs };
enum Weight { kPreGammaW, kPostGammaW, kGateW, kPostBetaW, kWeights };

// A weight of all rows, or nullptr where there is none (1, or for a beta 0).
__device__ __forceinline__ const float* weight_vector(const rowop_block_norm_args& a, int w)
{
    return w == kPreGammaW    ? (a.pre_norm != ROWOP_NORM_NONE ? a.pre_gamma : nullptr)
           : w == kPostGammaW ? (a.post_norm != ROWOP_NORM_NONE ? a.post_gamma : nullptr)
           : w == kPostBetaW  ? (a.post_norm == ROWOP_NORM_LAYER ? a.post_beta : nullptr)
                              : nullptr;
}

// The thread's group of row r's gate.
template <bool kPack, int NT, typename B>
__device__ __forceinline__ void gate_group(float (&v)[8], const rowop_block_norm_args& a, int64_t r, int lane, int off, int width)
{
    const int bytes = a.gate_type == GEMM_C_F32 ? 4 : sizeof(B);
    const char* gate = static_cast<const char*>(gate_row(a, r, bytes));
    load_gate<kPack, NT, B>(v, gate ? gate + static_cast<int64_t>(off) * bytes : nullptr, bytes == 4, lane, 0, width);
}

// A part's rows in order, with the sums over rows of the thread's own eight
// columns in registers. `at(v, input, r)` gives the thread's group of a
// matrix, `weight(v, w, r)` of a weight, `sums` adds over the row, `done(r)` is
// called when the row's inputs have been read. `off` is the first of the CTA's
// columns, `width` their number.
template <typename B, typename S, int NT, bool kPack, bool kBeta, typename At, typename WeightAt, typename Sums, typename Done>
__device__ __forceinline__ void backward_rows(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                                              int64_t part, int lane, int off, int width, At at, WeightAt weight, Sums sums,
                                              Done done)
{
    const float inv = 1.0f / static_cast<float>(a.width);
    const bool pre = a.pre_norm != ROWOP_NORM_NONE, post = a.post_norm != ROWOP_NORM_NONE;
    const bool pre_layer = a.pre_norm == ROWOP_NORM_LAYER, post_layer = a.post_norm == ROWOP_NORM_LAYER;
    const bool gate_f32 = a.gate_type == GEMM_C_F32;
    float acc[kBeta ? kSums : kPreBeta][8] = {};
    int64_t first, end;
    split.range(part, a.rows, first, end);
    int64_t flush = split.direct ? min((first / a.rows_per_gate + 1) * a.rows_per_gate, end) : end;
    // A row's statistics, read a row ahead: (mean, reciprocal deviation) before and after.
    auto stats = [&](int64_t r) {
        const int64_t i = 2 * min(r, end - 1);
        return make_float4(pre ? a.pre_stats[i] : 0.0f, pre ? a.pre_stats[i + 1] : 1.0f, post ? a.post_stats[i] : 0.0f,
                           post ? a.post_stats[i + 1] : 1.0f);
    };
    float4 ahead = first < end ? stats(first) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t r = first; r < end; ++r) {
        float d[8], t[8], w[8], hh[8], sum[2] = {0.0f, 0.0f};
        const float pre_mean = ahead.x, pre_rs = ahead.y, mean = ahead.z, rs = ahead.w;
        ahead = stats(r + 1);
        at(d, kDh, r);
        if (pre) {
            at(t, kDz, r);
            at(hh, kH, r);
            weight(w, kPreGammaW, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                hh[e] = (hh[e] - pre_mean) * pre_rs;  // of a column past the row's end: not 0, but t is
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
                d[e] += column<kPack, NT>(lane, 0, e) < width ? pre_rs * (t[e] - s0 - hh[e] * s1) : 0.0f;
        }
        if (g.dx) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = a.residual_scale * d[e];
            store_group<kPack, NT>(static_cast<S*>(g.dx) + r * g.lddx + off, t, lane, 0, width);
        }
        at(hh, kY, r);
        done(r);
        weight(w, kPostGammaW, r);
        if constexpr (kBeta) {
            weight(t, kPostBetaW, r);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            hh[e] = (hh[e] - mean) * rs;
            d[e] *= a.branch_scale;
            acc[kGate][e] = fmaf(d[e], fmaf(hh[e], w[e], t[e]), acc[kGate][e]);
        }
        weight(t, kGateW, r);
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
                const int64_t to = r / a.rows_per_gate * g.lddg + off;
                if (gate_f32)
                    store_group<kPack, NT>(static_cast<float*>(g.dgate) + to, acc[kGate], lane, 0, width);
                else
                    store_group<kPack, NT>(static_cast<B*>(g.dgate) + to, acc[kGate], lane, 0, width);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                acc[kGate][e] = 0.0f;
            flush = min(flush + a.rows_per_gate, end);
        }
    }
    float* out = static_cast<float*>(g.workspace) + part * split.sums * split.stride + off;
#pragma unroll
    for (int s = 0; s < (kBeta ? kSums : kPreBeta); ++s)
        store_group<kPack, NT>(out + s * split.stride, acc[s], lane, 0, width);
}

// Narrow rows: a warp a part, rows straight into registers.
template <typename B, typename S, bool kPack, bool kBeta>
__global__ void __launch_bounds__(128)
    sat_block_norm_backward_kernel(const __grid_constant__ rowop_block_norm_args a,
                                   const __grid_constant__ rowop_block_norm_grads g, const Split split)
{
    const int64_t part = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    if (part >= split.parts)
        return;
    const int lane = threadIdx.x % 32, width = static_cast<int>(a.width);
    int turn = 0;
    backward_rows<B, S, 32, kPack, kBeta>(
        a, g, split, part, lane, 0, width,
        [&](float(&v)[8], int input, int64_t r) {
            if (input == kDz)
                load_group<kPack, 32>(v, static_cast<const B*>(g.dz) + r * g.lddz, lane, 0, width);
            else if (input == kY)
                load_group<kPack, 32>(v, static_cast<const B*>(a.y) + r * a.ldy, lane, 0, width);
            else if (input == kH)
                load_group<kPack, 32>(v, static_cast<const S*>(a.h) + r * a.ldh, lane, 0, width);
            else if (g.dh)
                load_group<kPack, 32>(v, static_cast<const S*>(g.dh) + r * g.lddh, lane, 0, width);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = 0.0f;
        },
        [&](float(&v)[8], int w, int64_t r) {
            if (w == kGateW)
                gate_group<kPack, 32, B>(v, a, r, lane, 0, width);
            else
                load_weights<kPack, 32>(v, weight_vector(a, w), w == kPostBetaW ? 0.0f : 1.0f, lane, 0, width);
        },
        [&](float(&v)[2]) { row_sums<32>(v, nullptr, turn); }, [](int64_t) {});
}

// Wider rows: a CTA of NT threads a part, or a cluster of split.ctas, each of
// which takes NT 8 columns; rows through a ring, weights (and a gate that all
// rows share) kept in shared memory behind it. A cluster adds its CTAs' sums in
// order of rank: each sends its own to all, counted on a barrier.
template <typename B, typename S, int NT, bool kPack, bool kBeta>
__global__ void __launch_bounds__(NT + 32, 512 / NT)
    sat_block_norm_backward_ring_kernel(const __grid_constant__ rowop_block_norm_args a,
                                        const __grid_constant__ rowop_block_norm_grads g, const Split split, int stages,
                                        int stage_bytes)
{
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ __align__(8) Ring ring;
    __shared__ __align__(8) uint64_t arrived[2];
    __shared__ __align__(8) float2 across[2][kMaxCluster];
    __shared__ float scratch[2 * 2 * (NT / 32)];
    const int ctas = split.ctas, rank = blockIdx.x % ctas, lane = threadIdx.x;
    const int64_t part = blockIdx.x / ctas;
    const int off = rank * NT * 8, width = min(max(0, static_cast<int>(a.width) - off), NT * 8);
    auto source = [&](const void* p, int64_t ld, int bytes, int offset) {
        return Source{p ? static_cast<const char*>(p) + static_cast<int64_t>(off) * bytes : nullptr, ld * bytes, width * bytes, offset};
    };
    const bool pre = a.pre_norm != ROWOP_NORM_NONE;
    const int share = static_cast<int>(min(a.width, static_cast<int64_t>(NT * 8)));
    const int s_bytes = (share * static_cast<int>(sizeof(S)) + 31) / 16 * 16, b_bytes = (share * static_cast<int>(sizeof(B)) + 31) / 16 * 16;
    const Source sources[kInputs] = {source(g.dh, g.lddh, sizeof(S), 0), source(pre ? g.dz : nullptr, g.lddz, sizeof(B), 2 * s_bytes),
                                     source(pre ? a.h : nullptr, a.ldh, sizeof(S), s_bytes),
                                     source(a.y, a.ldy, sizeof(B), 2 * s_bytes + b_bytes)};
    constexpr int kept = kBeta ? kWeights : kPostBetaW;
    float* weights = reinterpret_cast<float*>(ring_memory + stages * stage_bytes);
    const bool shared_gate = !a.gate || a.rows_per_gate >= a.rows;
    for (int w = 0; w < kept; ++w)
        for (int c = threadIdx.x; c < width; c += NT + 32) {
            const float* v = weight_vector(a, w);
            float x = v ? v[off + c] : w == kPostBetaW ? 0.0f : 1.0f;
            if (w == kGateW && a.gate && shared_gate)
                x = a.gate_type == GEMM_C_F32 ? static_cast<const float*>(a.gate)[off + c] : to_f32(static_cast<const B*>(a.gate)[off + c]);
            weights[w * NT * 8 + c] = x;
        }
    for (int w = 0; w < kept; ++w)  // past the row's end: finite
        for (int c = width + threadIdx.x; c < NT * 8; c += NT + 32)
            weights[w * NT * 8 + c] = 0.0f;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&arrived[0]), 1);
        mbar_init(smem_u32(&arrived[1]), 1);
        ring.init(stages, NT / 32);
    }
    __syncthreads();
    if (ctas > 1)
        cluster_sync();  // all have started and have their barriers
    bool failed = false;
    int s = 0, round = 0, turn = 0, swaps = 0;
    auto next = [&] {
        if (++s == stages)
            s = 0, ++round;
    };
    if (threadIdx.x >= NT) {
        int64_t first, end;
        split.range(part, a.rows, first, end);
        for (int64_t r = first; r < end; ++r, next())
            ring.fill<kPack>(ring_memory + s * stage_bytes, s, round, sources, r, failed);
        return;
    }
    bool taken = false;
    backward_rows<B, S, NT, kPack, kBeta>(
        a, g, split, part, lane, off, width,
        [&](float(&v)[8], int input, int64_t r) {
            if (!taken)
                ring.take(s, round, failed);
            taken = true;
            const unsigned char* stage = ring_memory + s * stage_bytes;
            if (input == kDz || input == kY)
                stage_group<kPack, NT, B>(v, stage, sources[input], r, lane, 0, width);
            else if (sources[input].p)
                stage_group<kPack, NT, S>(v, stage, sources[input], r, lane, 0, width);
            else
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = 0.0f;
            if (failed)
                v[0] = NAN;
        },
        [&](float(&v)[8], int w, int64_t r) {
            if (w == kGateW && !shared_gate) {
                gate_group<kPack, NT, B>(v, a, r, lane, off, width);
            } else if constexpr (kPack) {
                const float4* at = reinterpret_cast<const float4*>(weights + w * NT * 8) + 2 * lane;
                const float4 x = at[0], y = at[1];
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = weights[w * NT * 8 + e * NT + lane];
            }
        },
        [&](float(&v)[2]) {
            ring_sums<NT>(v, scratch, turn);
            if (ctas > 1) {
                const int b = swaps & 1;
                if (threadIdx.x == 0)
                    mbar_arrive_expect_tx(smem_u32(&arrived[b]), ctas * 8);
                if (threadIdx.x < ctas)
                    send_b64(map_to_cta(smem_u32(&across[b][rank]), threadIdx.x), pair(v[0], v[1]),
                             map_to_cta(smem_u32(&arrived[b]), threadIdx.x));
                Ring::wait(&arrived[b], swaps >> 1 & 1, failed);
                ++swaps;
                v[0] = failed ? NAN : 0.0f, v[1] = 0.0f;
                for (int c = 0; c < ctas; ++c)
                    v[0] += across[b][c].x, v[1] += across[b][c].y;
            }
        },
        [&](int64_t) {
            ring.release(s);
            next();
            taken = false;
        });
}

template <typename B, typename S, int NT, bool kPack, bool kBeta>
cudaError_t launch_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    const int64_t share = a.width < NT * 8 ? a.width : NT * 8;
    const int stage = static_cast<int>(2 * ((share * sizeof(S) + 31) / 16 * 16) + 2 * ((share * sizeof(B) + 31) / 16 * 16));
    constexpr int room = kSmemPerSM / (512 / NT) - 2048, kept = (kBeta ? kWeights : kPostBetaW) * NT * 8 * 4;
    int stages = (room - kept) / stage;
    stages = stages < kMaxStages ? stages : kMaxStages;
    auto kernel = sat_block_norm_backward_ring_kernel<B, S, NT, kPack, kBeta>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel), room);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split.parts * split.ctas));
    cfg.blockDim = dim3(NT + 32);
    cfg.dynamicSmemBytes = stages * stage + kept;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split.ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, g, split, stages, stage);
}

template <typename B, typename S, bool kPack, bool kBeta>
cudaError_t choose_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    switch (backward_threads(a.width)) {
    case 32:
        sat_block_norm_backward_kernel<B, S, kPack, kBeta>
            <<<static_cast<unsigned>((split.parts + 3) / 4), 128, 0, s>>>(a, g, split);
        return cudaGetLastError();
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
