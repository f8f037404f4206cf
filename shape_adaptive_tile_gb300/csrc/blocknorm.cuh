// Block norm and its gradients (include/rowops.h): the kernels and their
// choice, instantiated for one type of the block in each blocknorm_<type>.cu.
//
// HBM bandwidth bounds both directions: every row is read once and written
// once. NT threads hold a row in registers, eight or more columns each. In
// rows that start on boundaries of eight elements (kPack) a thread's columns
// are groups of eight, moved by one 16- or 32-byte instruction; otherwise
// neighbouring threads hold neighbouring columns and move them one by one.
//
// Where there are more rows than CTAs, a CTA stays for many, with the next rows
// on their way into a ring in shared memory, so that memory does not wait for
// the reductions that each row has between its read and its write.
//
// Measured on a GB300, of its copy rate of 6.8 TB/s: forward 8192 x 8192 bf16
// 87 us (6.15 TB/s, 90%); 2049 x 5001 fp32, whose rows move four bytes at a
// time, 36 us (67%); backward 16384 x 4096 bf16 on an fp32 stream 206 us (5.87
// TB/s, 86%); 4593 x 1537 fp16 with Layer norms, whose elements move by
// themselves, 70 us (18%: the instructions bound it, 830 for a warp's 256 elements).
#pragma once

#include "blocknorm.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace sat {
namespace blocknorm {

using namespace rows;

// Eight elements as four pairs, on which the arithmetic goes two at a time.
struct Group {
    uint64_t p[4];
};

__device__ __forceinline__ uint64_t both(float v) { return pair(v, v); }

__device__ __forceinline__ Group fill(float v)
{
    return {{both(v), both(v), both(v), both(v)}};
}

template <typename T>
__device__ __forceinline__ Group group_of(const Pack<T>& v)
{
    Group g;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
            g.p[e] = pair(__uint_as_float(v.w[2 * e]), __uint_as_float(v.w[2 * e + 1]));
        } else {
            const float2 f = unpack2<T>(v.w[e]);
            g.p[e] = pair(f.x, f.y);
        }
    }
    return g;
}

// The thread's share of a row: column of its element e of group i.
template <bool kPack, int NT>
__device__ __forceinline__ int column(int lane, int i, int e)
{
    return kPack ? (i * NT + lane) * 8 + e : (i * 8 + e) * NT + lane;
}

// Group i of a row of `width` elements; columns from `width` on are 0.
template <bool kPack, int NT, typename T>
__device__ __forceinline__ Group load_group(const T* row, int lane, int i, int width)
{
    if constexpr (kPack) {
        const int c = column<true, NT>(lane, i, 0);
        return c < width ? group_of(load_pack(row + c)) : fill(0.0f);
    } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false, NT>(lane, i, e);
            v[e] = c < width ? to_f32(row[c]) : 0.0f;
        }
        return {{pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])}};
    }
}

template <bool kPack, int NT, typename T>
__device__ __forceinline__ void store_group(T* row, const Group& g, int lane, int i, int width)
{
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = halves(g.p[e]);
        v[2 * e] = f.x, v[2 * e + 1] = f.y;
    }
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

// The group with 0 in columns from `width` on.
template <bool kPack, int NT>
__device__ __forceinline__ Group inside(const Group& g, int lane, int i, int width)
{
    if constexpr (kPack) {
        return column<true, NT>(lane, i, 0) < width ? g : fill(0.0f);
    } else {
        Group o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = halves(g.p[e]);
            o.p[e] = pair(column<false, NT>(lane, i, 2 * e) < width ? f.x : 0.0f,
                          column<false, NT>(lane, i, 2 * e + 1) < width ? f.y : 0.0f);
        }
        return o;
    }
}

// A vector of weights, or `otherwise` where there is none.
template <bool kPack, int NT>
__device__ __forceinline__ Group load_weights(const float* w, float otherwise, int lane, int i, int width)
{
    return w ? load_group<kPack, NT>(w, lane, i, width) : fill(otherwise);
}

// A weight vector of `width` columns, or `otherwise`, into shared memory, with
// 0 behind it up to `room`; eight loads in flight a thread.
template <typename T>
__device__ __forceinline__ void keep_weights(float* to, const T* w, float otherwise, int width, int room)
{
    for (int c = threadIdx.x; c < room; c += 8 * blockDim.x) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = c + e * blockDim.x >= width ? 0.0f : w ? to_f32(w[c + e * blockDim.x]) : otherwise;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e * blockDim.x < room)
                to[c + e * blockDim.x] = v[e];
    }
}

// Group i of weights that lie in shared memory.
template <bool kPack, int NT>
__device__ __forceinline__ Group kept_group(const float* w, int lane, int i)
{
    if constexpr (kPack) {
        const ulonglong2* at = reinterpret_cast<const ulonglong2*>(w + column<true, NT>(lane, i, 0));
        const ulonglong2 x = at[0], y = at[1];
        return {{x.x, x.y, y.x, y.y}};
    } else {
        Group g;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            g.p[e] = pair(w[column<false, NT>(lane, i, 2 * e)], w[column<false, NT>(lane, i, 2 * e + 1)]);
        return g;
    }
}

// Puts the thread's first group there.
template <bool kPack, int NT>
__device__ __forceinline__ void keep_group(float* w, const Group& g, int lane)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = halves(g.p[e]);
        w[column<kPack, NT>(lane, 0, 2 * e)] = f.x;
        w[column<kPack, NT>(lane, 0, 2 * e + 1)] = f.y;
    }
}

__device__ __forceinline__ float sum_of(uint64_t v)
{
    const float2 f = halves(v);
    return f.x + f.y;
}

// The gate row of row r, by a 32-bit division (there are fewer than 2^31 rows); where there is a gate, as
// rows_per_gate may be 0 without one.
__device__ __forceinline__ int64_t gate_row(const rowop_block_norm_args& a, int64_t r)
{
    return a.rows_per_gate >= a.rows ? 0 : static_cast<uint32_t>(r) / static_cast<uint32_t>(a.rows_per_gate);
}

// The thread's group i of gate row k, in the gate's type: the block's or fp32
// (a branch that all threads take alike). `off`: the first column.
template <bool kPack, int NT, typename B>
__device__ __forceinline__ Group gate_group(const rowop_block_norm_args& a, int64_t k, int lane, int i, int off, int width)
{
    const int bytes = a.gate_type == GEMM_C_F32 ? 4 : sizeof(B);
    if (!a.gate)
        return fill(1.0f);
    const char* gate = static_cast<const char*>(a.gate) + (k * a.ldg + off) * bytes;
    if (bytes == 4)
        return load_group<kPack, NT>(reinterpret_cast<const float*>(gate), lane, i, width);
    return load_group<kPack, NT>(reinterpret_cast<const B*>(gate), lane, i, width);
}

// ---- rows through shared memory ------------------------------------------------------

constexpr int kMaxStages = 8;

// One of the matrices that a kernel reads row by row (none where p is NULL).
struct Source {
    const char* p;    // the CTA's first column of row 0
    int64_t pitch;    // bytes from row to row
    int bytes;        // of the CTA's share of a row
    int offset;       // where it lies in a stage

    __device__ __forceinline__ uint64_t row(int64_t r) const { return reinterpret_cast<uint64_t>(p + r * pitch); }
    // How many bytes after a 16-byte boundary it begins.
    __device__ __forceinline__ uint32_t begins(int64_t r) const
    {
        return (static_cast<uint32_t>(reinterpret_cast<uint64_t>(p)) + static_cast<uint32_t>(r) * static_cast<uint32_t>(pitch)) & 15;
    }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, uint64_t src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Groups of threads that may share a ring.
constexpr int kMaxGroups = 4;

// A ring of `stages` stages, each with a row of every source: filled by one
// warp (Ring::fill), read by `warps` others (Ring::take, Ring::release). Bulk
// copies move what lies between 16-byte boundaries of memory; where rows do
// not start on them (not kPack), a row lies in its stage as many bytes after
// a boundary as in memory, and the warp moves its ends by plain loads.
//
// Where groups of threads take the rows in turn, a stage is now one group's
// and now another's (unless the stages are a multiple of the groups). A wait
// tells a barrier's phases apart by their parity alone, so whoever waits has to
// see every one of them: each group has its own `full` barriers, on which only
// its own rows are counted. The filling warp waits for all of `empty`'s phases.
struct Ring {
    uint64_t full[kMaxGroups][kMaxStages], empty[kMaxStages];

    __device__ __forceinline__ void init(int stages, int warps)
    {
        for (int s = 0; s < stages; ++s) {
            for (int g = 0; g < kMaxGroups; ++g)
                mbar_init(smem_u32(&full[g][s]), 1);
            mbar_init(smem_u32(&empty[s]), warps);
        }
        fence_mbar_init();
    }

    static __device__ __forceinline__ void wait(uint64_t* bar, int parity, bool& failed)
    {
        failed = failed || !wait_bounded<true>(smem_u32(bar), parity);
    }

    // Returns whether it has: not where the stage does not become free.
    template <bool kPack, int N>
    __device__ __forceinline__ bool fill(unsigned char* stage, int s, int round, int group, const Source (&sources)[N], int64_t r)
    {
        uint64_t* const bar = &full[group][s];
        const int lane = threadIdx.x % 32;
        if (!__all_sync(0xffffffffu, wait_bounded<true>(smem_u32(&empty[s]), round & 1 ^ 1)))
            return false;
        uint32_t total = 0;
        if constexpr (kPack) {
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (sources[i].p && sources[i].bytes > 0)
                        total += sources[i].bytes;
                mbar_arrive_expect_tx(smem_u32(bar), total);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (sources[i].p && sources[i].bytes > 0)
                        bulk_load(smem_u32(stage) + sources[i].offset, sources[i].row(r), sources[i].bytes, smem_u32(bar));
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
                              smem_u32(bar));
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
                mbar_arrive_expect_tx(smem_u32(bar), total);
        }
        return true;
    }

    // The filling warp's last `stages` of `rows` rows for `groups` groups in turn: waits until they have landed.
    __device__ __forceinline__ void drain(int rows, int stages, int groups, int apart)
    {
        for (int k = max(0, rows - stages); k < rows; ++k)
            if (!wait_bounded<true, kDrainNs>(smem_u32(&full[k % groups][k % stages]), k / apart & 1))
                break;
    }

    // Waits for the use-th row that the group has had in stage s.
    __device__ __forceinline__ void take(int group, int s, int use, bool& failed) { wait(&full[group][s], use & 1, failed); }

    // The warp has read stage s: unless one of its lanes has given up, whose row may not have landed yet.
    __device__ __forceinline__ void release(int s, bool failed)
    {
        const bool read = !__any_sync(0xffffffffu, failed);
        __syncwarp();
        if (read && threadIdx.x % 32 == 0)
            mbar_arrive(smem_u32(&empty[s]));
    }
};

// Group i of a row of `width` elements that lies in a stage; columns from `width` on are 0.
template <bool kPack, int NT, typename T>
__device__ __forceinline__ Group stage_group(const unsigned char* stage, const Source& source, int64_t r, int lane, int i, int width)
{
    if constexpr (kPack) {
        const int c = column<true, NT>(lane, i, 0);
        if (c >= width)
            return fill(0.0f);
        const uint4* at = reinterpret_cast<const uint4*>(stage + source.offset + c * sizeof(T));
        if constexpr (sizeof(T) == 4) {
            const uint4 x = at[0], y = at[1];
            return group_of(Pack<T>{{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}});
        } else {
            const uint4 x = at[0];
            return group_of(Pack<T>{{x.x, x.y, x.z, x.w}});
        }
    } else {
        const T* at = reinterpret_cast<const T*>(stage + source.offset + source.begins(r));
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = column<false, NT>(lane, i, e);
            v[e] = c < width ? to_f32(at[c]) : 0.0f;
        }
        return {{pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7])}};
    }
}

// Sums of N values (a power of two, at most 8) over NT threads of a CTA (the
// `group`-th NT), to each of them, in a fixed order, behind a barrier of theirs.
// Lanes halve the values that they hold while they double the lanes that
// those are of, so that eight sums take nine exchanges and not forty.
// `scratch`: 2 x N x NT / 32 floats; its halves take turns, so one barrier
// does: a half is written again two reductions later.
template <int NT, int N>
__device__ __forceinline__ void ring_sums(float (&v)[N], float* scratch, int& turn, int group)
{
    constexpr int W = NT / 32;
    static_assert((N & (N - 1)) == 0 && N <= 8 && W * N >= 4, "");
    const int warp = (threadIdx.x >> 5) % W, lane = threadIdx.x & 31;
    int n = N, bit = 16;
#pragma unroll
    for (; n > 1; n /= 2, bit /= 2) {
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = upper ? v[i] : v[i + n / 2], keep = upper ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
        }
    }
#pragma unroll
    for (; bit > 0; bit /= 2)
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
    // Lanes l with the same l / (32 / N) hold the sum whose number is that.
    float* half = scratch + turn * (N * W);
    turn ^= 1;
    if (lane % (32 / N) == 0)
        half[warp * N + lane / (32 / N)] = v[0];
    named_bar_sync(1 + group, NT);
    // Lane l: sum l % N of warps l / N, l / N + 32 / N, ...
    constexpr int each = 32 / N;  // warps that the lanes read at once
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; w += each)
        if (w + lane / N < W)
            s += half[(w + lane / N) * N + lane % N];
#pragma unroll
    for (int o = 16; o >= N; o /= 2)
        s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = __shfl_sync(0xffffffffu, s, i);
}

// Sums of K values over a cluster's CTAs, in order of rank: each sends its own
// to all, counted on a barrier there. `turn` counts the exchanges; `across` and
// `arrived` of the exchange before are still in use.
template <int K, int MAX>
__device__ __forceinline__ void cluster_sums(float (&v)[K], float (&across)[2][MAX][8], uint64_t (&arrived)[2], int thread, int rank,
                                             int ctas, int& turn, bool& failed)
{
    const int b = turn & 1;
    if (thread == 0 && !failed)
        mbar_arrive_expect_tx(smem_u32(&arrived[b]), ctas * ((K + 1) / 2) * 8);
    if (thread < ctas && !failed) {
        const uint32_t bar = map_to_cta(smem_u32(&arrived[b]), thread), to = map_to_cta(smem_u32(&across[b][rank][0]), thread);
#pragma unroll
        for (int k = 0; k < K; k += 2)
            send_b64(to + 4 * k, pair(v[k], k + 1 < K ? v[k + 1] : 0.0f), bar);
    }
    Ring::wait(&arrived[b], turn >> 1 & 1, failed);
    ++turn;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.0f;
        for (int c = 0; c < ctas; ++c)
            v[k] += across[b][c][k];
    }
}

// The end of a kernel whose CTAs wait. No CTA of a cluster ends while another
// may still send to it. Where this thread has given up, copies that it has
// started and sums that were sent to it before the barrier may be on their way,
// with nothing here that counts them any more: they have the time that a wait
// has, again.
__device__ __forceinline__ void end_of_rows(bool clustered, bool failed)
{
    if (clustered)
        cluster_sync();
    if (failed)
        for (const uint64_t since = globaltimer_ns(); globaltimer_ns() - since < kSettleNs;)
            ;
}

// ---- forward -----------------------------------------------------------------------

enum Weight { kPreGammaW, kPostGammaW, kGateW, kPreBetaW, kPostBetaW, kWeights };

// A weight of all rows, or nullptr where there is none (1, or for a beta 0).
__device__ __forceinline__ const float* weight_vector(const rowop_block_norm_args& a, int w)
{
    return w == kPreGammaW    ? (a.pre_norm != ROWOP_NORM_NONE ? a.pre_gamma : nullptr)
           : w == kPostGammaW ? (a.post_norm != ROWOP_NORM_NONE ? a.post_gamma : nullptr)
           : w == kPreBetaW   ? (a.pre_norm == ROWOP_NORM_LAYER ? a.pre_beta : nullptr)
           : w == kPostBetaW  ? (a.post_norm == ROWOP_NORM_LAYER ? a.post_beta : nullptr)
                              : nullptr;
}

// Mean and reciprocal deviation of a row of `whole` columns, of which NT
// threads hold `width` as NV groups each and `sums` adds up all. The
// variance is summed from the deviations, after the mean: the difference of
// two large sums would lose what rows far from 0 have of it. Without a Layer
// norm the mean is 0, and columns past the row's end hold 0 and add nothing.
template <bool kLayer, bool kPack, int NT, int NV, typename Sums>
__device__ __forceinline__ void moments(const Group (&v)[NV], int whole, int width, int kind, float eps, int lane, Sums sums,
                                        float& mean, float& r)
{
    const float inv = 1.0f / static_cast<float>(whole);
    mean = 0.0f;
    uint64_t q = 0;
    if (kLayer && kind == ROWOP_NORM_LAYER) {
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s = add2(s, v[i].p[e]);
        float total[1] = {sum_of(s)};
        sums(total);
        mean = total[0] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Group d;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d.p[e] = add2(v[i].p[e], both(-mean));
            d = inside<kPack, NT>(d, lane, i, width);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q = fma2(d.p[e], d.p[e], q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q = fma2(v[i].p[e], v[i].p[e], q);
    }
    float total[1] = {sum_of(q)};
    sums(total);
    r = 1.0f / sqrtf(total[0] * inv + eps);
}

// v = (v - mean) r gamma + beta
template <bool kLayer, typename WeightAt>
__device__ __forceinline__ void apply(Group& v, float mean, float r, WeightAt weight, int gamma, int beta, int i)
{
    const Group g = weight(gamma, i);
    const uint64_t r2 = both(r);
    if constexpr (kLayer) {
        const Group b = weight(beta, i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v.p[e] = fma2(mul2(add2(v.p[e], both(-mean)), r2), g.p[e], b.p[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v.p[e] = mul2(mul2(v.p[e], r2), g.p[e]);
    }
}

// What follows a row's read: v is y's share, x(i) gives x's groups, weight(w,
// i) a weight's; writes h, z and the statistics. `lane` is the thread's place
// among the NT that hold columns off .. off + width - 1 of the row.
template <typename B, typename S, int NT, int NV, bool kPack, bool kLayer, typename X, typename WeightAt, typename Sums>
__device__ __forceinline__ void finish_row(const rowop_block_norm_args& a, int64_t r, Group (&v)[NV], int lane, int off, int width,
                                           X x, WeightAt weight, Sums sums)
{
    const int whole = static_cast<int>(a.width);
    float mean, rs;
    if (a.post_norm != ROWOP_NORM_NONE) {
        moments<kLayer, kPack, NT, NV>(v, whole, width, a.post_norm, a.post_eps, lane, sums, mean, rs);
        if (a.post_stats && lane == 0 && off == 0)
            a.post_stats[2 * r] = mean, a.post_stats[2 * r + 1] = rs;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            apply<kLayer>(v[i], mean, rs, weight, kPostGammaW, kPostBetaW, i);
    }
    S* h = static_cast<S*>(a.h) + r * a.ldh + off;
    const uint64_t residual = both(a.residual_scale), branch = both(a.branch_scale);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Group u = x(i);
        if (a.gate) {
            const Group g = weight(kGateW, i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[i].p[e] = mul2(v[i].p[e], g.p[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[i].p[e] = fma2(residual, u.p[e], mul2(branch, v[i].p[e]));
        if (kLayer)
            v[i] = inside<kPack, NT>(v[i], lane, i, width);
        store_group<kPack, NT>(h, v[i], lane, i, width);
    }
    if (a.pre_norm == ROWOP_NORM_NONE)
        return;
    moments<kLayer, kPack, NT, NV>(v, whole, width, a.pre_norm, a.pre_eps, lane, sums, mean, rs);
    if (a.pre_stats && lane == 0 && off == 0)
        a.pre_stats[2 * r] = mean, a.pre_stats[2 * r + 1] = rs;
    B* z = static_cast<B*>(a.z) + r * a.ldz + off;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        apply<kLayer>(v[i], mean, rs, weight, kPreGammaW, kPreBetaW, i);
        store_group<kPack, NT>(z, v[i], lane, i, width);
    }
}

// Few rows, or narrow ones that a warp holds: rows straight into registers.
template <typename B, typename S, int NT, int NV, bool kPack, bool kLayer>
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
        Group v[NV], u[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = load_group<kPack, NT>(y, lane, i, width);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            u[i] = load_group<kPack, NT>(x, lane, i, width);
        // With one group a thread, the weights too are read before the first reduction.
        constexpr bool kEarly = NV == 1;
        Group early[kEarly ? kWeights : 1];
        auto read = [&](int w, int i) {
            return w == kGateW ? (a.gate ? gate_group<kPack, NT, B>(a, gate_row(a, r), lane, i, 0, width) : fill(1.0f))
                               : load_weights<kPack, NT>(weight_vector(a, w), w >= kPreBetaW ? 0.0f : 1.0f, lane, i, width);
        };
        if constexpr (kEarly) {
#pragma unroll
            for (int w = 0; w < (kLayer ? kWeights : kPreBetaW); ++w)
                early[w] = read(w, 0);
        }
        finish_row<B, S, NT, NV, kPack, kLayer>(
            a, r, v, lane, 0, width, [&](int i) { return u[i]; },
            [&](int w, int i) {
                if constexpr (kEarly)
                    return early[w];
                else
                    return read(w, i);
            },
            [&](float(&s)[1]) { row_sums<NT>(s, scratch, turn); });
    }
}

// Many rows: a CTA of 512 threads an SM, in groups of NT that each take a row
// at a time and share a ring of `stages` stages of `stage_bytes` and, behind it
// (`kept`), the weights. So several rows are at hand in an SM at once, one
// group's reductions beside another's arithmetic, with one copy of the weights.
// Rows past 8192 columns have a pair of CTAs (C = 2), half of the columns each.
template <typename B, typename S, int NT, int NV, int C, bool kPack, bool kLayer>
__global__ void __launch_bounds__(512 + 32, 1)
    sat_block_norm_ring_kernel(const __grid_constant__ rowop_block_norm_args a, int stages, int stage_bytes, bool kept)
{
    constexpr int G = 512 / NT;
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ __align__(8) Ring ring;
    __shared__ float scratch[G][2 * (NT / 32)];
    __shared__ __align__(8) uint64_t arrived[G][2];
    __shared__ __align__(8) float across[G][2][2][8];
    constexpr int room = NT * NV * 8;
    const int rank = blockIdx.x % C, off = rank * room, width = min(static_cast<int>(a.width) - off, room);
    const int y_bytes = (min(static_cast<int>(a.width), room) * static_cast<int>(sizeof(B)) + 31) / 16 * 16;
    const Source sources[2] = {{reinterpret_cast<const char*>(static_cast<const B*>(a.y) + off), a.ldy * static_cast<int64_t>(sizeof(B)),
                                width * static_cast<int>(sizeof(B)), 0},
                               {reinterpret_cast<const char*>(static_cast<const S*>(a.x) + off), a.ldx * static_cast<int64_t>(sizeof(S)),
                                width * static_cast<int>(sizeof(S)), y_bytes}};
    float* weights = reinterpret_cast<float*>(ring_memory + stages * stage_bytes);
    const bool shared_gate = a.gate && a.rows_per_gate >= a.rows;
    // Kept weights lie one after another in the order of Weight, those that the call does not have left out.
    const float* at[kWeights];
    int n = 0;
#pragma unroll
    for (int w = 0; w < kWeights; ++w) {
        const bool there = kept && (w == kGateW ? shared_gate : weight_vector(a, w) != nullptr);
        at[w] = there ? weights + n * room : nullptr;
        if (there && w == kGateW && a.gate_type != GEMM_C_F32)
            keep_weights(weights + n * room, static_cast<const B*>(a.gate) + off, 1.0f, width, room);
        else if (there)
            keep_weights(weights + n * room, (w == kGateW ? static_cast<const float*>(a.gate) : weight_vector(a, w)) + off, 1.0f, width, room);
        n += there;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < G; ++i) {
            mbar_init(smem_u32(&arrived[i][0]), 1);
            mbar_init(smem_u32(&arrived[i][1]), 1);
        }
        ring.init(stages, NT / 32);
    }
    __syncthreads();
    if (C > 1)
        cluster_sync();  // both have started and have their barriers
    const int64_t pair_of = blockIdx.x / C, pairs = gridDim.x / C;
    // The rows that a group has in one stage are as far apart, counted in the CTA's rows, as the least number that is a
    // multiple of both the stages and the groups.
    int apart = stages;
    while (apart % G)
        apart += stages;
    bool failed = false;
    int s = 0, round = 0, turn = 0;
    if (threadIdx.x >= 512) {
        int filling = 0, filled = 0;  // the group whose row it is, and the rows so far
        for (int64_t r = pair_of; r < a.rows; r += pairs, ++filled) {
            if (!ring.fill<kPack>(ring_memory + s * stage_bytes, s, round, filling, sources, r))
                break;
            if (++s == stages)
                s = 0, ++round;
            filling = filling + 1 == G ? 0 : filling + 1;
        }
        ring.drain(filled, stages, G, apart);
        end_of_rows(C > 1, false);
        return;
    }
    const int group = threadIdx.x / NT, lane = threadIdx.x % NT;
    // The group's k-th row of the CTA's: k = group, group + G, ...
    int use = 0, swaps = 0;
    s = group % stages;
    int k = group, next_use = apart;
    for (int64_t r = pair_of + group * pairs; r < a.rows; r += G * pairs, k += G, s = (s + G) % stages) {
        if (k >= next_use)
            ++use, next_use += apart;
        ring.take(group, s, use, failed);
        const unsigned char* stage = ring_memory + s * stage_bytes;
        Group v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = stage_group<kPack, NT, B>(stage, sources[0], r, lane, i, width);
        if (failed)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                v[i] = fill(NAN);
        finish_row<B, S, NT, NV, kPack, kLayer>(
            a, r, v, lane, off, width,
            [&](int i) {
                const Group u = stage_group<kPack, NT, S>(stage, sources[1], r, lane, i, width);
                if (i == NV - 1)
                    ring.release(s, failed);
                return u;
            },
            [&](int w, int i) {
                if (at[w])
                    return kept_group<kPack, NT>(at[w], lane, i);
                if (w == kGateW)
                    return gate_group<kPack, NT, B>(a, gate_row(a, r), lane, i, off, width);
                const float* vector = weight_vector(a, w);
                return load_weights<kPack, NT>(vector ? vector + off : nullptr, w >= kPreBetaW ? 0.0f : 1.0f, lane, i, width);
            },
            [&](float(&v)[1]) {
                ring_sums<NT>(v, scratch[group], turn, group);
                if constexpr (C > 1) {
                    cluster_sums(v, across[group], arrived[group], lane, rank, C, swaps, failed);
                    if (failed)
                        v[0] = NAN;
                }
            });
    }
    end_of_rows(C > 1, C > 1 && failed);
}

template <typename B, typename S, int NT, int NV, bool kPack, bool kLayer>
cudaError_t launch_forward(const rowop_block_norm_args& a, cudaStream_t s)
{
    const int64_t ctas = NT == 32 ? (a.rows + 3) / 4 : a.rows;
    sat_block_norm_kernel<B, S, NT, NV, kPack, kLayer>
        <<<static_cast<unsigned>(ctas < (1 << 20) ? ctas : (1 << 20)), NT == 32 ? 128 : NT, 0, s>>>(a);
    return cudaGetLastError();
}

// What a ring's CTA has in shared memory, for `columns` columns and groups of NT threads.
struct RingRoom {
    static constexpr int bytes = kSmemPerSM - 2048;
    int stage, weights;
    bool kept;  // the weights stay on chip: a row for every group and one more fit beside them
};

template <typename B, typename S>
RingRoom ring_room(const rowop_block_norm_args& a, int columns, int groups)
{
    const int64_t w = a.width < columns ? a.width : columns;
    const bool post = a.post_norm != ROWOP_NORM_NONE, pre = a.pre_norm != ROWOP_NORM_NONE;
    const int vectors = (post && a.post_gamma) + (pre && a.pre_gamma) + (a.gate && a.rows_per_gate >= a.rows) +
                        (a.post_norm == ROWOP_NORM_LAYER && a.post_beta) + (a.pre_norm == ROWOP_NORM_LAYER && a.pre_beta);
    RingRoom r;
    r.stage = static_cast<int>((w * sizeof(B) + 31) / 16 * 16 + (w * sizeof(S) + 31) / 16 * 16);
    r.weights = vectors * columns * 4;
    r.kept = RingRoom::bytes - r.weights >= (groups + 1) * r.stage;
    return r;
}

template <typename B, typename S, int NT, int NV, int C, bool kPack, bool kLayer>
cudaError_t launch_ring(const rowop_block_norm_args& a, cudaStream_t s)
{
    const RingRoom r = ring_room<B, S>(a, NT * NV * 8, 512 / NT);
    const int stage = r.stage, weights = r.kept ? r.weights : 0;
    int stages = (RingRoom::bytes - weights) / stage;
    stages = stages < kMaxStages ? stages : kMaxStages;
    if (stages < 1)
        return cudaErrorInvalidConfiguration;
    auto kernel = sat_block_norm_ring_kernel<B, S, NT, NV, C, kPack, kLayer>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel), RingRoom::bytes);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(kSMs / C * C));
    cfg.blockDim = dim3(512 + 32);
    cfg.dynamicSmemBytes = stages * stage + weights;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, stages, stage, r.kept);
}

// Whether rows of over 1024 columns go through the ring, not to a CTA each,
// whose threads hold a row with room for a second CTA's in the SM: by their
// number an SM and by what lies in a stage, x's and y's columns of one CTA.
// Large stages leave few in flight; weights that do not fit beside them, and
// gates that change, are read again for every row. A CTA a row pays more where
// elements move by themselves (not kPack) and for the Layer norm's further
// reductions. Measured in us, a CTA a row | the ring, inputs from HBM; b bf16,
// h fp16, f fp32, m bf16 on an fp32 stream, RMS norms and a shared gate where
// nothing else is said:
//   2048 b: 304 rows 4.6 | 6.3, 456 7.1 | 6.7, 4864 43 | 21; f: 456 7.9 | 7.8, 912 12.1 | 10.5
//   4096 b: 760 11.5 | 11.3, 1216 15.0 | 13.7, 4864 49 | 32; f: 608 11.3 | 12.1, 912 15.6 | 15.1; m: 912 14.1 | 13.7
//   6144 b: 1216 20.0 | 20.1, 1520 23.3 | 22.3, 4864 60 | 51; f: 1520 29.3 | 30.3, 4864 76 | 88; m: 1520 26.2 | 25.3;
//   b, a gate a row: 1520 29.2 | 32.6, 2432 43.8 | 47.7
//   8192 b: 1520 25.8 | 25.9, 2128 33.5 | 32.3, 4864 67 | 61; f: 4864 96 | 125; m: 4864 78 | 112
//   12288 b: 304 15.4 | 15.8, 456 19.9 | 19.1, 4864 135 | 104; f: 456 25.9 | 23.1, 4864 177 | 171; m: 4864 155 | 120
//   16384 b: 380 23.9 | 20.1, 4864 170 | 121; m: 4864 212 | 231; f without weights: 4864 186 | 210
//   Layer b: 2048 304 8.7 | 8.8, 608 14.7 | 9.9, 4096 608 15.7 | 12.7, 8192 1216 28 | 38, 16384 456 34.0 | 33.3; f: 4096 608
//   16.8 | 15.0, 12288 304 25.3 | 22.4, 2432 141 | 124
//   not kPack: 1537 b 1216 13.2 | 13.9, 2432 24.6 | 22.1; 3255 h 1216 16.4 | 16.4, a gate a row 22.9 | 19.3 (b 16.2 | 19.7);
//   6001 b 304 9.0 | 11.3, 456 15.1 | 13.1; 8001 f 2432 65 | 75; 12001 f 304 21 | 18, 2432 128 | 82; 16001 f 304 25.5 | 25.9,
//   2432 155 | 144; Layer b 1281 304 7.8 | 9.0, 608 14.1 | 11.3, 3001 608 16.0 | 14.3, 8001 2432 68 | 82
template <typename B, typename S, bool kPack, bool kLayer>
bool ring_pays(const rowop_block_norm_args& a)
{
    const int64_t rows = a.rows, w = a.width;
    const RingRoom r = ring_room<B, S>(a, w <= 2048 ? 2048 : w <= 4096 ? 4096 : w <= 6144 || (w > 8192 && w <= 12288) ? 6144 : 8192,
                                       w <= 4096 ? 4 : 2);
    if (w <= 4096)
        return rows >= (kLayer ? 4 : !kPack ? 8 : w <= 2048 ? 3 : 6) * kSMs;
    if (w > 8192)
        return kLayer ? rows >= 3 * kSMs : !kPack ? rows >= 2 * kSMs : rows >= 3 * kSMs && r.kept && r.stage <= 49 * 1024;
    if (!kPack)
        return rows >= 3 * kSMs && r.kept;
    return rows >= 10 * kSMs && r.kept && r.stage <= 40 * 1024 && (!a.gate || a.rows_per_gate >= a.rows);
}

template <typename B, typename S, bool kPack, bool kLayer>
cudaError_t choose_forward_as(const rowop_block_norm_args& a, cudaStream_t s)
{
    // Few rows, and rows of up to 1024 columns: a CTA a row and as many threads as it has groups (4864 x 1024 bf16 13.1 us, in
    // the ring 15.1). In the ring two to four groups a thread, so that a row's fixed work (the reductions, its addresses) is
    // spread over up to 32 columns; three where that is enough (4864 x 5120 bf16 50 us, with four 57; 10240 103 | 119).
    if (a.width <= 256)
        return launch_forward<B, S, 32, 1, kPack, kLayer>(a, s);
    if (a.width <= 1024)
        return launch_forward<B, S, 128, 1, kPack, kLayer>(a, s);
    if (!ring_pays<B, S, kPack, kLayer>(a))
        return a.width <= 4096   ? launch_forward<B, S, 512, 1, kPack, kLayer>(a, s)
               : a.width <= 8192 ? launch_forward<B, S, 512, 2, kPack, kLayer>(a, s)
                                 : launch_forward<B, S, 512, 4, kPack, kLayer>(a, s);
    if (a.width <= 2048)
        return launch_ring<B, S, 128, 2, 1, kPack, kLayer>(a, s);
    if (a.width <= 4096)
        return launch_ring<B, S, 128, 4, 1, kPack, kLayer>(a, s);
    if (a.width <= 6144)
        return launch_ring<B, S, 256, 3, 1, kPack, kLayer>(a, s);
    if (a.width <= 8192)
        return launch_ring<B, S, 256, 4, 1, kPack, kLayer>(a, s);
    if (a.width <= 12288)
        return launch_ring<B, S, 256, 3, 2, kPack, kLayer>(a, s);
    return launch_ring<B, S, 256, 4, 2, kPack, kLayer>(a, s);
}

template <typename B, typename S, bool kPack>
cudaError_t choose_forward(const rowop_block_norm_args& a, cudaStream_t s)
{
    return a.post_norm == ROWOP_NORM_LAYER || a.pre_norm == ROWOP_NORM_LAYER ? choose_forward_as<B, S, kPack, true>(a, s)
                                                                             : choose_forward_as<B, S, kPack, false>(a, s);
}

// ---- backward ----------------------------------------------------------------------

// The sources of the backward pass.
enum Input { kDh, kDz, kH, kY, kInputs };

// A part's rows in order, with the sums over rows of the thread's own eight
// columns in registers. With t = dz gamma_pre, u = dh + r_pre t, hh and yh the
// normed h and y and w = branch_scale gate gamma_post, the gradient of h is
//
//   D = u - r_pre (s0 + hh s1),   s1 = mean(t hh),  s0 = mean(t) (Layer)
//
// and the second norm's means, of w D yh and (Layer) w D, are linear in s0 and
// s1: the sums that they are made of need nothing of the first norm, so a row
// has one reduction and not two in turn. Columns past the row's end have
// weights of 0 and gradients of 0.
//
// `at(input, r)` gives the thread's group of a matrix, `weight(w)` of a weight
// and `gate()` of the gate, whose row `change_gate(k)` makes the k-th; `sums`
// adds over the row once its inputs have been read, `done()` ends it; `failed()` says at the end whether a row's inputs
// did not come. `off` is the first of the CTA's columns, `width` their number.
template <typename B, typename S, int NT, int NV, bool kPack, int MODE, typename At, typename WeightAt, typename GateAt,
          typename ChangeGate, typename Sums, typename Done, typename Failed>
__device__ __forceinline__ void backward_rows(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                                              int64_t part, int lane, int off, int width, At at, WeightAt weight, GateAt gate,
                                              ChangeGate change_gate, Sums sums, Done done, Failed failed)
{
    constexpr bool kBeta = MODE != kRms, kGrouped = MODE == kLayerGrouped;
    const float inv = 1.0f / static_cast<float>(a.width);
    const bool pre = a.pre_norm != ROWOP_NORM_NONE, post = a.post_norm != ROWOP_NORM_NONE;
    const bool pre_layer = a.pre_norm == ROWOP_NORM_LAYER, post_layer = a.post_norm == ROWOP_NORM_LAYER;
    const uint64_t branch = both(a.branch_scale), residual = both(a.residual_scale);
    // Sums over rows of dz hh, D yh and, for betas, dz, D. A gate that all rows
    // share multiplies these at the end; one that changes, at its last row, into
    // sums of gate D yh and gate D: registers, or (Layer) the part's own place
    // in the workspace, where each thread adds up its own columns.
    const bool grouped = kGrouped || (MODE == kRms && a.gate && a.rows_per_gate < a.rows);
    Group dz_hh[NV], d_yh[NV], gd_yh[NV], dz_1[NV], d_1[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        dz_hh[i] = d_yh[i] = gd_yh[i] = dz_1[i] = d_1[i] = fill(0.0f);
    int64_t first, end;
    split.range(part, a.rows, first, end);
    float* out = static_cast<float*>(g.workspace) + part * split.sums * split.stride + off;
    auto own = [&](int sum, int i) { return load_group<kPack, NT>(out + sum * split.stride, lane, i, width); };
    auto put = [&](int sum, int i, const Group& v) { store_group<kPack, NT>(out + sum * split.stride, v, lane, i, width); };
    if (kGrouped)
#pragma unroll
        for (int i = 0; i < NV; ++i)
            put(kPostGamma, i, fill(0.0f)), put(kPostBeta, i, fill(0.0f));
    // A row's statistics, read a row ahead: (mean, reciprocal deviation) before and after.
    auto stats = [&](int64_t r) {
        const int64_t i = 2 * min(r, end - 1);
        return make_float4(pre ? a.pre_stats[i] : 0.0f, pre ? a.pre_stats[i + 1] : 1.0f, post ? a.post_stats[i] : 0.0f,
                           post ? a.post_stats[i + 1] : 1.0f);
    };
    // The gradient of the gate, of sums over its rows.
    auto gate_grad = [&](int i) {
        const Group gamma = weight(kPostGammaW, i), beta = kBeta ? weight(kPostBetaW, i) : fill(0.0f);
        Group o;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o.p[e] = mul2(branch, kBeta ? fma2(gamma.p[e], d_yh[i].p[e], mul2(beta.p[e], d_1[i].p[e])) : mul2(gamma.p[e], d_yh[i].p[e]));
        return o;
    };
    // The sums with the gate, of what has come since its row began.
    auto gate_ends = [&](int i) {
        const Group gr = gate(i);
        if constexpr (kGrouped) {
            Group yh = own(kPostGamma, i), one = own(kPostBeta, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                yh.p[e] = fma2(mul2(branch, gr.p[e]), d_yh[i].p[e], yh.p[e]);
                one.p[e] = fma2(mul2(branch, gr.p[e]), d_1[i].p[e], one.p[e]);
            }
            put(kPostGamma, i, yh), put(kPostBeta, i, one);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                gd_yh[i].p[e] = fma2(mul2(branch, gr.p[e]), d_yh[i].p[e], gd_yh[i].p[e]);
        }
    };
    // The gate row at hand and the row after its last.
    int64_t gate_at = grouped ? first / a.rows_per_gate : 0, gate_end = grouped ? (gate_at + 1) * a.rows_per_gate : end;
    if (first < end)
        change_gate(gate_at);
    S* dx = static_cast<S*>(g.dx) + first * g.lddx + off;
    B* dy = static_cast<B*>(g.dy) + first * g.lddy + off;
    float4 ahead = first < end ? stats(first) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t r = first; r < end; ++r, dx += g.lddx, dy += g.lddy) {
        const float4 st = ahead;
        ahead = stats(r + 1);
        const uint64_t pre_rs = both(st.y), rs = both(st.w);
        Group u[NV], hh[NV], yh[NV], w[NV];
        uint64_t s[kBeta ? 8 : 4] = {};  // the fourth of four is not used
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            u[i] = at(kDh, r, i), yh[i] = at(kY, r, i), w[i] = weight(kPostGammaW, i), hh[i] = fill(0.0f);
            Group dz = fill(0.0f);
            if (pre) {
                dz = at(kDz, r, i);
                hh[i] = at(kH, r, i);
                const Group gamma = weight(kPreGammaW, i);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (kBeta)
                        hh[i].p[e] = add2(hh[i].p[e], both(-st.x));
                    hh[i].p[e] = mul2(hh[i].p[e], pre_rs);
                    dz_hh[i].p[e] = fma2(dz.p[e], hh[i].p[e], dz_hh[i].p[e]);
                    if constexpr (kBeta)
                        dz_1[i].p[e] = add2(dz_1[i].p[e], dz.p[e]);
                    dz.p[e] = mul2(dz.p[e], gamma.p[e]);
                    u[i].p[e] = fma2(dz.p[e], pre_rs, u[i].p[e]);
                }
            }
            const Group gr = gate(i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kBeta)
                    yh[i].p[e] = add2(yh[i].p[e], both(-st.z));
                yh[i].p[e] = mul2(yh[i].p[e], rs);
                w[i].p[e] = mul2(mul2(w[i].p[e], branch), gr.p[e]);
                const uint64_t c = mul2(w[i].p[e], yh[i].p[e]);
                s[0] = fma2(dz.p[e], hh[i].p[e], s[0]);
                s[1] = fma2(c, u[i].p[e], s[1]);
                s[2] = fma2(c, hh[i].p[e], s[2]);
                if constexpr (kBeta) {
                    s[3] = add2(s[3], dz.p[e]);
                    s[4] = add2(s[4], c);
                    s[5] = fma2(w[i].p[e], u[i].p[e], s[5]);
                    s[6] = add2(s[6], w[i].p[e]);
                    s[7] = fma2(w[i].p[e], hh[i].p[e], s[7]);
                }
            }
        }
        constexpr int K = kBeta ? 8 : 4;
        float sum[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            sum[k] = sum_of(s[k]);
        sums(sum);
        done();
        const float s1 = sum[0] * inv, s0 = kBeta && pre_layer ? sum[3] * inv : 0.0f;
        float e1 = sum[1] - st.y * s1 * sum[2], e0 = 0.0f;
        if constexpr (kBeta) {
            e1 -= st.y * s0 * sum[4];
            e0 = post_layer ? (sum[5] - st.y * (s0 * sum[6] + s1 * sum[7])) * inv : 0.0f;
        }
        e1 = post ? e1 * inv : 0.0f;
        const uint64_t h_by = both(-st.y * s1), h_less = both(-st.y * s0), y_by = both(-e1), y_less = both(-e0);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[i].p[e] = fma2(hh[i].p[e], h_by, u[i].p[e]);
                if constexpr (kBeta)
                    u[i].p[e] = add2(u[i].p[e], h_less);
            }
            if (kBeta && pre_layer)
                u[i] = inside<kPack, NT>(u[i], lane, i, width);
            Group o;
            if (g.dx) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o.p[e] = mul2(residual, u[i].p[e]);
                store_group<kPack, NT>(dx, o, lane, i, width);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d_yh[i].p[e] = fma2(u[i].p[e], yh[i].p[e], d_yh[i].p[e]);
                if constexpr (kBeta)
                    d_1[i].p[e] = add2(d_1[i].p[e], u[i].p[e]);
                o.p[e] = fma2(yh[i].p[e], y_by, mul2(w[i].p[e], u[i].p[e]));
                if constexpr (kBeta)
                    o.p[e] = add2(o.p[e], y_less);
                o.p[e] = mul2(o.p[e], rs);
            }
            if (g.dy)
                store_group<kPack, NT>(dy, o, lane, i, width);
        }
        if (grouped && (r + 1 == gate_end || r + 1 == end)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                gate_ends(i);
                if (split.direct) {  // the part has all of the gate row's rows
                    if (g.dgate && a.gate_type == GEMM_C_F32)
                        store_group<kPack, NT>(static_cast<float*>(g.dgate) + gate_at * g.lddg + off, gate_grad(i), lane, i, width);
                    else if (g.dgate)
                        store_group<kPack, NT>(static_cast<B*>(g.dgate) + gate_at * g.lddg + off, gate_grad(i), lane, i, width);
                }
                if (r + 1 < end)  // without the gate's gradient a part may go on from one gate row to the next
                    d_yh[i] = d_1[i] = fill(0.0f);
            }
            if (r + 1 < end) {
                change_gate(++gate_at);
                gate_end += a.rows_per_gate;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (failed())  // the rows' sums have made the others NaN
            dz_hh[i] = dz_1[i] = fill(NAN);
        if (!grouped)
            gate_ends(i);
        put(kPreGamma, i, dz_hh[i]);
        put(kGate, i, gate_grad(i));
        if constexpr (!kGrouped)
            put(kPostGamma, i, gd_yh[i]);
        if constexpr (kBeta)
            put(kPreBeta, i, dz_1[i]);
        if constexpr (MODE == kLayerShared) {
            const Group gr = gate(i);
            Group o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o.p[e] = mul2(mul2(branch, gr.p[e]), d_1[i].p[e]);
            put(kPostBeta, i, o);
        }
    }
}

// Narrow rows: a warp a part, rows straight into registers.
template <typename B, typename S, bool kPack, int MODE>
__global__ void __launch_bounds__(128)
    sat_block_norm_backward_kernel(const __grid_constant__ rowop_block_norm_args a,
                                   const __grid_constant__ rowop_block_norm_grads g, const Split split)
{
    const int64_t part = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    if (part >= split.parts)
        return;
    const int lane = threadIdx.x % 32, width = static_cast<int>(a.width);
    int turn = 0;
    Group gate_now = fill(0.0f);
    backward_rows<B, S, 32, 1, kPack, MODE>(
        a, g, split, part, lane, 0, width,
        [&](int input, int64_t r, int) {
            return input == kDz  ? load_group<kPack, 32>(static_cast<const B*>(g.dz) + r * g.lddz, lane, 0, width)
                   : input == kY ? load_group<kPack, 32>(static_cast<const B*>(a.y) + r * a.ldy, lane, 0, width)
                   : input == kH ? load_group<kPack, 32>(static_cast<const S*>(a.h) + r * a.ldh, lane, 0, width)
                   : g.dh        ? load_group<kPack, 32>(static_cast<const S*>(g.dh) + r * g.lddh, lane, 0, width)
                                 : fill(0.0f);
        },
        [&](int w, int) {
            return inside<kPack, 32>(load_weights<kPack, 32>(weight_vector(a, w), w >= kPreBetaW ? 0.0f : 1.0f, lane, 0, width),
                                     lane, 0, width);
        },
        [&](int) { return gate_now; }, [&](int64_t k) { gate_now = gate_group<kPack, 32, B>(a, k, lane, 0, 0, width); },
        [&](auto& v) { row_sums<32>(v, nullptr, turn); }, [] {}, [] { return false; });
}

// Wider rows: a CTA of NT threads a part, or a cluster of split.ctas, each of
// which takes NT 8 columns; rows through a ring, weights (and a gate that all
// rows share) kept in shared memory behind it. A cluster adds its CTAs' sums in
// order of rank: each sends its own to all, counted on a barrier.
//
// The ring here has no warp of its own, which would take registers from all:
// the barrier in a row's reduction says that all have read the row before, and
// then thread 0 sends for the row that goes in its place. The ends of rows
// that do not start on 16-byte boundaries are read by the first 64 threads, a
// two-byte piece each, at the start of a row and written at its end.
template <typename B, typename S, int NT, bool kPack, int MODE>
__global__ void __launch_bounds__(NT, kBackwardPerSM<NT>)
    sat_block_norm_backward_ring_kernel(const __grid_constant__ rowop_block_norm_args a,
                                        const __grid_constant__ rowop_block_norm_grads g, const Split split, int stages,
                                        int stage_bytes)
{
    extern __shared__ __align__(128) unsigned char ring_memory[];
    __shared__ __align__(8) uint64_t full[kMaxStages], arrived[2];
    __shared__ __align__(8) float across[2][kMaxCluster][8];
    __shared__ float scratch[2 * 8 * (NT / 32)];
    constexpr bool kBeta = MODE != kRms;
    constexpr int room = NT * 8;
    const int ctas = split.ctas, rank = blockIdx.x % ctas, lane = threadIdx.x;
    const int64_t part = blockIdx.x / ctas;
    const int off = rank * room, width = min(max(0, static_cast<int>(a.width) - off), room);
    auto source = [&](const void* p, int64_t ld, int bytes, int offset) {
        return Source{p ? static_cast<const char*>(p) + static_cast<int64_t>(off) * bytes : nullptr, ld * bytes, width * bytes, offset};
    };
    const bool pre = a.pre_norm != ROWOP_NORM_NONE;
    const int share = static_cast<int>(min(a.width, static_cast<int64_t>(room)));
    const int s_bytes = (share * static_cast<int>(sizeof(S)) + 31) / 16 * 16, b_bytes = (share * static_cast<int>(sizeof(B)) + 31) / 16 * 16;
    const Source sources[kInputs] = {source(g.dh, g.lddh, sizeof(S), 0), source(pre ? g.dz : nullptr, g.lddz, sizeof(B), 2 * s_bytes),
                                     source(pre ? a.h : nullptr, a.ldh, sizeof(S), s_bytes),
                                     source(a.y, a.ldy, sizeof(B), 2 * s_bytes + b_bytes)};
    // Kept: gamma before, gamma after, the gate and (Layer) the beta after.
    float* weights = reinterpret_cast<float*>(ring_memory + stages * stage_bytes);
    const bool shared_gate = !a.gate || a.rows_per_gate >= a.rows;
    auto vector_of = [&](int w) { return weight_vector(a, w) ? weight_vector(a, w) + off : nullptr; };
    keep_weights(weights, vector_of(kPreGammaW), 1.0f, width, room);
    keep_weights(weights + room, vector_of(kPostGammaW), 1.0f, width, room);
    if (a.gate && shared_gate && a.gate_type != GEMM_C_F32)
        keep_weights(weights + 2 * room, static_cast<const B*>(a.gate) + off, 1.0f, width, room);
    else
        keep_weights(weights + 2 * room, a.gate && shared_gate ? static_cast<const float*>(a.gate) + off : nullptr, 1.0f, width, room);
    if (kBeta)
        keep_weights(weights + 3 * room, vector_of(kPostBetaW), 0.0f, width, room);
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&arrived[0]), 1);
        mbar_init(smem_u32(&arrived[1]), 1);
        for (int s = 0; s < stages; ++s)
            mbar_init(smem_u32(&full[s]), kPack ? 1 : 3);
        fence_mbar_init();
    }
    __syncthreads();
    if (ctas > 1)
        cluster_sync();  // all have started and have their barriers

    int64_t first, end;
    split.range(part, a.rows, first, end);
    // Thread 0: row r's bulk copies into stage s.
    auto send = [&](int64_t r, int s) {
        unsigned char* stage = ring_memory + s * stage_bytes;
        uint32_t total = 0;
#pragma unroll
        for (int i = 0; i < kInputs; ++i) {
            const uint64_t lo = sources[i].row(r), hi = lo + sources[i].bytes, lo16 = (lo + 15) & ~15ull, hi16 = hi & ~15ull;
            if (!sources[i].p || hi16 <= lo16)
                continue;
            const uint32_t bytes = static_cast<uint32_t>(hi16 - lo16);
            total += bytes;
            bulk_load(smem_u32(stage) + sources[i].offset + static_cast<uint32_t>(lo16 - (lo & ~15ull)), lo16, bytes, smem_u32(&full[s]));
        }
        mbar_arrive_expect_tx(smem_u32(&full[s]), total);
    };
    // Threads 0 .. 63: this thread's piece of row r's ends: its address (0 for none) and its place in a stage.
    const int input = lane / 16 % kInputs, piece = lane % 16;
    const Source mine = input == kDh ? sources[kDh] : input == kDz ? sources[kDz] : input == kH ? sources[kH] : sources[kY];
    auto end_of = [&](int64_t r, int& place) -> uint64_t {
        const uint64_t lo = mine.row(r), hi = lo + mine.bytes, lo16 = (lo + 15) & ~15ull, hi16 = hi & ~15ull;
        const uint64_t x = (piece < 8 ? lo & ~15ull : hi16) + piece % 8 * 2;
        place = mine.offset + static_cast<int>(x - (lo & ~15ull));
        return mine.p && x >= lo && x < hi && (x < lo16 || x >= hi16) && (piece < 8 || hi16 >= lo16) ? x : 0;
    };
    bool failed = false;
    auto put_end = [&](int s, int place, uint64_t x, uint16_t v) {
        const bool sure = !__any_sync(0xffffffffu, failed);
        if (x)
            *reinterpret_cast<uint16_t*>(ring_memory + s * stage_bytes + place) = v;
        __syncwarp();
        if (sure && lane % 32 == 0)
            mbar_arrive(smem_u32(&full[s]));
    };
    for (int s = 0; s < stages && first + s < end; ++s) {
        if (threadIdx.x == 0)
            send(first + s, s);
        if (!kPack && threadIdx.x < 64) {
            int place;
            const uint64_t x = end_of(first + s, place);
            put_end(s, place, x, x ? *reinterpret_cast<const uint16_t*>(x) : 0);
        }
    }

    bool taken = false;
    int s = 0, round = 0, turn = 0, swaps = 0, place = 0;
    uint64_t x = 0;
    uint16_t held = 0;
    int64_t now = first;  // the row at hand
    backward_rows<B, S, NT, 1, kPack, MODE>(
        a, g, split, part, lane, off, width,
        [&](int in, int64_t r, int) {
            if (!taken) {
                // The row that will take the place of the one before.
                const int64_t ahead = r - 1 + stages;
                if (!kPack && threadIdx.x < 64 && r > first && ahead < end) {
                    x = end_of(ahead, place);
                    held = x ? *reinterpret_cast<const uint16_t*>(x) : 0;
                }
                Ring::wait(&full[s], round & 1, failed);
                taken = true;
            }
            const unsigned char* stage = ring_memory + s * stage_bytes;
            return in == kDz || in == kY ? stage_group<kPack, NT, B>(stage, sources[in], r, lane, 0, width)
                   : sources[in].p       ? stage_group<kPack, NT, S>(stage, sources[in], r, lane, 0, width)
                                         : fill(0.0f);
        },
        [&](int w, int) { return kept_group<kPack, NT>(weights + (w == kPreGammaW ? 0 : w == kPostGammaW ? 1 : 3) * room, lane, 0); },
        [&](int) { return kept_group<kPack, NT>(weights + 2 * room, lane, 0); },
        [&](int64_t k) {  // each thread its own columns: nobody else reads them
            if (!shared_gate)
                keep_group<kPack, NT>(weights + 2 * room, gate_group<kPack, NT, B>(a, k, lane, 0, off, width), lane);
        },
        [&](auto& v) {
            if (!kPack && threadIdx.x < 64)
                fence_proxy_async_smem();  // of the ends written before: what follows them there comes by bulk copies
            if (failed)  // with its sum the row's gradients are NaN, all of them
                v[0] = NAN;
            ring_sums<NT>(v, scratch, turn, 0);
            const int before = s == 0 ? stages - 1 : s - 1;
            if (now > first && now - 1 + stages < end) {
                if (threadIdx.x == 0 && !failed)
                    send(now - 1 + stages, before);
                if (!kPack && threadIdx.x < 64)
                    put_end(before, place, x, held);
            }
            if (ctas > 1)
                cluster_sums(v, across, arrived, threadIdx.x, rank, ctas, swaps, failed);
            if (failed)
                v[0] = NAN;
        },
        [&] {
            taken = false;
            ++now;
            if (++s == stages)
                s = 0, ++round;
        },
        [&] { return failed; });
    end_of_rows(ctas > 1, failed);
}

template <typename B, typename S, int NT, bool kPack, int MODE>
cudaError_t launch_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    const int64_t share = a.width < NT * 8 ? a.width : NT * 8;
    const int stage = static_cast<int>(2 * ((share * sizeof(S) + 31) / 16 * 16) + 2 * ((share * sizeof(B) + 31) / 16 * 16));
    constexpr int room = kSmemPerSM / kBackwardPerSM<NT> - 3072, kept = (MODE == kRms ? 3 : 4) * NT * 8 * 4;
    int stages = (room - kept) / stage;
    stages = stages < kMaxStages ? stages : kMaxStages;
    if (stages < 2)
        return cudaErrorInvalidConfiguration;
    auto kernel = sat_block_norm_backward_ring_kernel<B, S, NT, kPack, MODE>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel), room);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split.parts * split.ctas));
    cfg.blockDim = dim3(NT);
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

template <typename B, typename S, bool kPack, int MODE>
cudaError_t choose_backward(const rowop_block_norm_args& a, const rowop_block_norm_grads& g, const Split& split,
                            cudaStream_t s)
{
    switch (split.threads) {
    case 32:
        sat_block_norm_backward_kernel<B, S, kPack, MODE>
            <<<static_cast<unsigned>((split.parts + 3) / 4), 128, 0, s>>>(a, g, split);
        return cudaGetLastError();
    case 128: return launch_backward<B, S, 128, kPack, MODE>(a, g, split, s);
    case 256: return launch_backward<B, S, 256, kPack, MODE>(a, g, split, s);
    default: return launch_backward<B, S, 512, kPack, MODE>(a, g, split, s);
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
    switch (split.mode) {
    case kRms: return pack ? choose_backward<B, S, true, kRms>(a, g, split, s) : choose_backward<B, S, false, kRms>(a, g, split, s);
    case kLayerShared:
        return pack ? choose_backward<B, S, true, kLayerShared>(a, g, split, s) : choose_backward<B, S, false, kLayerShared>(a, g, split, s);
    default:
        return pack ? choose_backward<B, S, true, kLayerGrouped>(a, g, split, s) : choose_backward<B, S, false, kLayerGrouped>(a, g, split, s);
    }
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
