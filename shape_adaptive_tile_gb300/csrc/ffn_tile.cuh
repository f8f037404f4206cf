// The tile kernel of the feed-forward operators: tcgen05 products of 16-bit or
// microscaled 4-bit operands whose epilogue is the activation and the product
// of two projections, their gradient, or a plain store.
//
// Roles as in the GEMM kernel: one warp fills a ring of shared-memory stages by
// TMA, one thread issues the MMAs, eight warps take the accumulators from
// tensor memory to the outputs. Two kinds of launch:
//   - persistent (one CTA or CTA pair an SM or SM pair): tiles in grouped raster
//     order, two accumulators in turn so that a tile's epilogue runs beside the
//     next one's products (16-bit operands; the scales of 4-bit ones leave room
//     for one accumulator of 256 columns);
//   - split: one tile a cluster, whose CTAs take a share of k each and add their
//     sums through distributed shared memory in rank order. For problems of few
//     tiles, and for a few tokens (swap: the weights are the first operand, their
//     outputs the accumulator's rows, and the tokens its 16 to 64 columns).
// A gated tile holds the same columns of both projections: as halves of its
// columns (in a pair, each CTA loads one half), or, swapped, as two accumulators.
//
// What bounds them, and what they take:
//   - 16-bit pairs' tiles: the tensor pipe, 87% busy (2048 x 4096 to 2 x 8192, 144 us), and, back to back, the power: 8192 x
//     4096 to 2 x 16384 in 1230 us, 1.79 PFLOP/s. Of outputs off 16 bytes the epilogue: 2047 x 1000 to 2 x 2501 with the
//     pre-activations 34 us, the tensor pipe 26% busy.
//   - 4-bit pairs' tiles: 600 cycles a stage, of which the products are 512 at four times the rate of 16 bits and the loads
//     from L2 436 when nothing else runs (8192 of k); what keeps both from running side by side has not been measured, the
//     products of a stage waiting for the next stage's scales is one candidate. Then the drain of the one accumulator:
//     8192 x 8192 x 8192 in 185 us, 5.9 PFLOP/s.
//   - a few tokens: memory. One token, 4096 to 2 x 16384, in 45 us, 6.0 TB/s; 48 tokens, 2048 to 2 x 8192, in 17 us, of which 5
//     are the launch, the first loads and the last stores.
//   - shared 128 x 128 tiles: loads, 0.22 us for a stage of 32 KB a CTA, then the sums' way between the CTAs, 0.8 us and 0.65
//     for each of them: 515 x 4006 by 1001 as 120 CTAs 14 us.
#pragma once

#include <atomic>
#include <type_traits>

#include "ffn_ptx.cuh"
#include "ffn_tile.h"

namespace sat {
namespace ffn {

template <bool MX_, int EPI_, int CG_, int BN_, bool P_MN_, bool Q_MN_, bool SWAP_, bool SPLIT_>
struct TileTraits {
    static constexpr bool MX = MX_, P_MN = P_MN_, Q_MN = Q_MN_, SWAP = SWAP_, SPLIT = SPLIT_;
    static constexpr int EPI = EPI_, CG = CG_, BN = BN_;
    static constexpr bool GATED = EPI != kStore;
    static constexpr int BK = MX ? 256 : 64;              // k of one stage: rows of 128 bytes
    static constexpr int NP = SWAP && GATED ? 2 : 1;      // first operands a stage
    static constexpr int P_BYTES = 128 * 128;
    static constexpr int BN_CTA = BN / CG;                // second operand's rows this CTA loads
    static constexpr int Q_BYTES = BN_CTA * 128;
    static constexpr int QBOX = BN_CTA < 64 ? BN_CTA : 64;  // rows (or columns, MN-major) of one box
    // Scales of a stage: two words (of four blocks of 32) for each row: 1 KB for 128 rows.
    static constexpr int NQT = (BN + 127) / 128;          // row tiles of the second operand's scales
    static constexpr int SF_BYTES = MX ? 1024 * (NP + NQT) : 0;
    static constexpr int STAGE_BYTES = NP * P_BYTES + Q_BYTES + SF_BYTES;
    static constexpr int TX_BYTES = STAGE_BYTES;
    static constexpr int EPI_WARPS = 8;
    static constexpr int EPI_BYTES = SWAP ? 0 : EPI_WARPS * 4096;
    static constexpr int BAR_BYTES = 512;
    // Two CTAs an SM for few tokens (their prologues and ends overlap), else one.
    static constexpr int BUDGET = (SWAP && BN <= 32 ? 113 : 227) * 1024 - 1024 - EPI_BYTES - BAR_BYTES - (SWAP && BN <= 32 ? 1024 : 0);
    static constexpr int STAGES = BUDGET / STAGE_BYTES > 8 ? 8 : BUDGET / STAGE_BYTES;
    static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + EPI_BYTES + BAR_BYTES;
    static constexpr int THREADS = (2 + EPI_WARPS) * 32;
    static constexpr int ACC_COLS = NP * BN;
    static constexpr int ACCS = SPLIT || (MX && BN > 128) ? 1 : 2;
    static constexpr bool DRAIN = !SPLIT && (MX || EPI == kGated);  // an accumulator is taken to registers at once
    // Scale columns of a stage: 4 for each of two words of 128 rows.
    static constexpr int SF_COLS = MX ? 8 * (NP + NQT) : 0;
    static constexpr int NEED_COLS = ACCS * ACC_COLS + STAGES * SF_COLS;
    static constexpr int TMEM_COLS = NEED_COLS <= 32 ? 32 : NEED_COLS <= 64 ? 64 : NEED_COLS <= 128 ? 128 : NEED_COLS <= 256 ? 256 : 512;
    // Columns of one epilogue step, counted in output columns.
    static constexpr int CHUNK = SWAP ? 16 : SPLIT ? 32 : 64;
    static constexpr int OUT_COLS = GATED && !SWAP ? BN / 2 : BN;  // output columns of a tile (swapped: tokens)
    static constexpr int NCHUNK = OUT_COLS / CHUNK;
    static constexpr int CHUNK_ACC = GATED ? 2 * CHUNK : CHUNK;    // accumulator columns of a chunk
    static constexpr int PART_BYTES = CHUNK_ACC * 128 * 4;         // a chunk's partial sums of one CTA
    // The output columns of a tile that each half of the epilogue warps has: whole chunks in turn, or, drained, one half of them.
    static constexpr int RUN = DRAIN ? OUT_COLS / 2 : CHUNK, RUNS = OUT_COLS / RUN;

    static_assert(!MX || (!P_MN && !Q_MN), "4-bit operands are K-major");
    static_assert(!SWAP || (SPLIT && CG == 1 && !Q_MN), "few tokens: split, K-major tokens");
    static_assert(!SPLIT || CG == 1, "split tiles are 1-SM");
    static_assert(!DRAIN || BN == 256, "half the tile's columns a warp");
    static_assert(EPI != kGrad || !SWAP, "no swapped gradient");
    static_assert(OUT_COLS % CHUNK == 0, "whole chunks");
    static_assert(STAGES >= 2 && NEED_COLS <= 512, "ring or tensor memory");
    static_assert((SWAP && BN <= 32 ? 2 : 1) * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
    // CTAs of a kernel and of one beside it may meet on an SM, and the later ones wait for the earlier ones' end: whatever
    // fits there together has to find its tensor memory together. One of more than 151 KB meets none of 75.5 KB or more
    // (with 1 KB of the system's each).
    static_assert(SMEM_BYTES > 151 * 1024 || (SMEM_BYTES >= 75 * 1024 + 512 && TMEM_COLS <= 128), "tensor memory of an SM");
};

// 1 / x to a unit in the last place, of x from 1 to 2^126 (one instruction).
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 2^x to 2^-22 of it, of x from -126 to 126 (one instruction).
__device__ __forceinline__ float power_of_two(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(by x), of by x from -150 to 0: the square of a power of two with half the exponent, which is no number below the normal
// ones where the result is. kFine: by (x + low), and what the exponent's roundings (its own and the constant's) left out comes
// in as a factor 1 + ... . Without it the result is off by up to 2^-23.7 of itself times by x (and 2^-24 times by x where x
// was rounded): 1.2e-5 at most where an fp32 result ends, which an output rounded to 16 bits (2^-9 or 2^-12) does not show. It
// is for fp32 outputs: 4-bit gated 2049 x 4096 x 8200 to fp16 took 68.7 us with it and 66.6 without, gradients recomputed 2048
// x 1024 x 4096 96.1 and 94.0.
template <bool kFine>
__device__ __forceinline__ float exp_product(float x, float low, double by)
{
    const double factor = 0.72134752044448170 * by;  // log2(e) / 2
    const float c = static_cast<float>(factor), rest = static_cast<float>(factor - c);
    const float y = c * x;
    const float e = power_of_two(y);
    if constexpr (!kFine)
        return e * e;
    const float off = fmaf(rest, x, fmaf(c, low, fmaf(c, x, -y)));
    return fmaf(1.3862943611198906f * off, e, e) * e;
}

// s = 1 / (1 + exp(-x)) and o = 1 - s, each with a small error relative to itself: from exp(-|x|), which does not overflow.
// (Left of -87 a quotient by 1 + exp(-x) is 0 or lost where s is a number yet.)
template <bool kFine>
__device__ __forceinline__ void logistic(float x, float& s, float& o)
{
    const float e = exp_product<kFine>(fminf(fabsf(x), 150.0f), 0.0f, -1.0);
    const float r = reciprocal(1.0f + e);
    s = x < 0.0f ? e * r : r;
    o = x < 0.0f ? r : e * r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int kind);

// a(g) and a'(g) of the activation KIND (ffn_activation_t), for outputs in fp32 (kFine) or of 16 bits.
template <int KIND, bool kFine>
__device__ __forceinline__ void act_grad(float g, float& a, float& d)
{
    if constexpr (KIND == 1) {
        float s, o;
        logistic<kFine>(g, s, o);
        a = g * s;
        d = s * fmaf(g, o, 1.0f);
    } else if constexpr (KIND == 2) {
        // The normal distribution's integral below -x as its density phi(x) times the Mills ratio, which is smooth: t P(t)
        // with t = 1 / (1 + 0.27 x), the form of Hastings, Approximations for Digital Computers, with coefficients of this
        // file's own, fitted by least squares reweighted to the smallest relative error, 2.5e-8 for x from 0 to 16. Below 0 the
        // activation is that tail itself, so its error has to be relative too, some 20 of fp32's half steps. (From 14.5 on phi
        // is 0 in fp32; infinities stay out of the products.) The derivative wants phi too.
        const float x = fminf(fabsf(g), 16.0f);
        const float t = reciprocal(fmaf(0.27f, x, 1.0f));
        const float h = x * x;
        const float phi = 0.39894228040143268f * exp_product<kFine>(h, fmaf(x, x, -h), -0.5);
        float q = fmaf(0.0727893636f, t, -0.318029493f);
        q = fmaf(q, t, 0.427678317f);
        q = fmaf(q, t, -0.175963894f);
        q = fmaf(q, t, 0.272060841f);
        q = fmaf(q, t, 0.179808944f);
        q = fmaf(q, t, 0.255413711f);
        q = fmaf(q, t, 0.26953879f);
        q = fmaf(q, t, 0.270017594f);
        q *= t * phi;
        const float c = g < 0.0f ? q : 1.0f - q;
        a = g * c;
        d = fmaf(g, phi, c);
    } else if constexpr (KIND == 3) {  // (1 + tanh y) / 2 = 1 / (1 + exp(-2 y))
        float s, o;
        logistic<kFine>(1.5957691216057308f * fmaf(0.044715f * g * g, g, g), s, o);
        a = g * s;
        // (g^2 is held to what no s (1 - s) but 0 meets, or it would overflow to 0 times infinity.)
        d = fmaf(a * o, 1.5957691216057308f * fmaf(0.134145f, fminf(g * g, 1e6f), 1.0f), s);
    } else if constexpr (KIND == 4) {
        a = g > 0.0f ? g : (g != g ? g : 0.0f);
        d = g > 0.0f ? 1.0f : (g != g ? g : 0.0f);
    } else {
        a = g;
        d = 1.0f;
    }
}

// f(std::integral_constant<int, kind>): the choice is made once for a whole
// loop over values. Made for each of 64 unrolled values instead, the code ran
// to tens of kilobytes, whose fetching took a single tile's epilogue 9 us.
template <class F>
__device__ __forceinline__ void with_act(int kind, F f)
{
    if (kind == 1)
        f(std::integral_constant<int, 1>{});
    else if (kind == 2)
        f(std::integral_constant<int, 2>{});
    else if (kind == 3)
        f(std::integral_constant<int, 3>{});
    else if (kind == 4)
        f(std::integral_constant<int, 4>{});
    else
        f(std::integral_constant<int, 0>{});
}

// g = a(g) u
template <bool kFine, int N>
__device__ __forceinline__ void gate_as(float (&g)[N], const float (&u)[N], int kind)
{
    with_act(kind, [&](auto k) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float a, d;
            act_grad<decltype(k)::value, kFine>(g[j], a, d);
            g[j] = a * u[j];
        }
    });
}

// (fp32 outputs: of 4-bit operands only)
template <class T, int N>
__device__ __forceinline__ void gate(float (&g)[N], const float (&u)[N], int kind, int out_kind)
{
    if (T::MX && out_kind == 0)
        gate_as<true>(g, u, kind);
    else
        gate_as<false>(g, u, kind);
}

__device__ __forceinline__ void unpack2(uint32_t v, int kind, float& lo, float& hi);

// From gate g, other factor u and dh (pairs of 16-bit elements): g = dg, u = du.
__device__ __forceinline__ void slope(float (&g)[32], float (&u)[32], const uint32_t (&dh)[16], int kind, int activation)
{
    with_act(activation, [&](auto k) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float d[2];
            unpack2(dh[j], kind, d[0], d[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float a, s;
                act_grad<decltype(k)::value, false>(g[2 * j + e], a, s);
                g[2 * j + e] = d[e] * u[2 * j + e] * s;
                u[2 * j + e] = d[e] * a;
            }
        }
    });
}

// N elements of one kind, `step` apart (16-bit kinds rounded to nearest even), for those of index below n.
template <int N>
__device__ __forceinline__ void store_column(void* at, int kind, long long first, long long step, int n, const float (&v)[N])
{
    if (kind == 0) {
        float* o = static_cast<float*>(at) + first;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n)
                o[j * step] = v[j];
    } else {
        uint16_t* o = static_cast<uint16_t*>(at) + first;
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const uint32_t w = pack2(v[j], v[j + 1], kind);
            if (j < n)
                o[j * step] = static_cast<uint16_t>(w);
            if (j + 1 < n)
                o[(j + 1) * step] = static_cast<uint16_t>(w >> 16);
        }
    }
}

// Two floats rounded to bf16 (kind 1) or fp16 (kind 2), the first in the lower half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int kind)
{
    uint32_t r;
    if (kind == 1)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack2(uint32_t v, int kind, float& lo, float& hi)
{
    if (kind == 1) {
        lo = __uint_as_float(v << 16);
        hi = __uint_as_float(v & 0xFFFF0000u);
    } else {
        const __half2 h = *reinterpret_cast<const __half2*>(&v);
        const float2 f = __half22float2(h);
        lo = f.x;
        hi = f.y;
    }
}

// Waits are bounded: a whole warp's, each of at most kWaitNs. Who gives up raises
// the CTA's abort flag (and a pair's other CTA's), and every wait that is not over
// then gives up too. Nothing more is loaded, multiplied or released after that, so
// no stage is filled and no barrier armed out of turn; outputs whose sums have not
// come are NaN; and the CTA ends only after the limit again (2 ms at least), when
// whatever was on its way has landed. The clock is read only after a few tries: a
// ring whose stages are used up as fast as they come waits at every one of them.
#ifndef SAT_FFN_WAIT_NS
#define SAT_FFN_WAIT_NS 2000000000ull
#endif
constexpr unsigned long long kWaitNs = SAT_FFN_WAIT_NS;
// (try_wait may suspend a thread for longer than a limit below this, which only tests have.)
constexpr bool kSuspend = kWaitNs >= 1000000;
constexpr int kWaitTries = kSuspend ? 64 : 0, kWaitRound = kSuspend ? 32 : 1;

struct Waiter {
    uint32_t abort;       // shared address of the flag
    uint32_t peer_abort;  // the same of the pair's other CTA, or of this one

    __device__ __forceinline__ bool aborted() const { return ld_shared_u32(abort) != 0; }
};

// Of a whole warp: true or false in all lanes.
template <bool kCluster>
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, const Waiter w)
{
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        bool there = false;
        for (int i = 0; i < kWaitRound && !there; ++i)
            there = kSuspend ? mbar_try_wait<kCluster>(bar, parity) : mbar_test_wait<kCluster>(bar, parity);
        if (__all_sync(0xffffffffu, there))
            return true;
        if (__any_sync(0xffffffffu, w.aborted()))
            return false;
        if (__any_sync(0xffffffffu, globaltimer_ns() - t0 >= kWaitNs)) {
            st_shared_u32(w.abort, 1u);
            if (w.peer_abort != w.abort)
                st_cluster_u32(w.peer_abort, 1u);
            return false;
        }
    }
}

template <bool kCluster>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, const Waiter& w)
{
    bool there = false;
#pragma unroll 1
    for (int i = 0; i < kWaitTries && !there; ++i)
        there = mbar_try_wait<kCluster>(bar, parity);
    return __all_sync(0xffffffffu, there) || wait_long<kCluster>(bar, parity, w);
}

static __device__ __noinline__ void wait_again()
{
    const uint64_t t0 = globaltimer_ns(), ns = kWaitNs > 2000000ull ? kWaitNs : 2000000ull;
    while (globaltimer_ns() - t0 < ns)
        __nanosleep(1000);
}

// 16-bit rows start, start + STEP, ... of a staged chunk, all of which start on
// a word (ODD false) or all between two words (ODD): then a lane's second
// element and the next lane's first make a word. (A store costs the same some four
// cycles of the SM whatever it moves, so the rows' ends are left to two stores
// for all rows together.)
template <bool ODD, int STEP>
__device__ __forceinline__ void store_words(uint32_t sb, uint16_t* out, long long ld, int start, int rows, int n)
{
    const int lane = threadIdx.x & 31;
    uint32_t at[8 / STEP], next[8 / STEP];
#pragma unroll
    for (int i = 0; i < 8 / STEP; ++i) {
        const int r = (start + i * STEP) & 7;
        at[i] = sb + r * 128 + ((((lane >> 2) ^ r) << 4) | ((lane & 3) << 2));
        const int l1 = min(lane + 1, 31);
        next[i] = sb + r * 128 + ((((l1 >> 2) ^ r) << 4) | ((l1 & 3) << 2));
    }
    const int e = 2 * lane + (ODD ? 1 : 0);  // first element of this lane's word
    const bool word = e + 1 < n;
    const long long step = static_cast<long long>(STEP) * ld;
    uint16_t* o = out + start * ld;
#pragma unroll 1
    for (int r0 = start; r0 < rows; r0 += 8) {
        uint32_t v[8 / STEP], w[8 / STEP];
#pragma unroll
        for (int i = 0; i < 8 / STEP; ++i) {
            v[i] = ld_shared_u32(at[i]);
            w[i] = ODD ? ld_shared_u32(next[i]) : 0u;
            at[i] += 1024;
            next[i] += 1024;
        }
#pragma unroll
        for (int i = 0; i < 8 / STEP; ++i, o += step) {
            if (ODD)
                w[i] = __funnelshift_r(v[i], w[i], 16);
            else
                w[i] = v[i];
            if (r0 + i * STEP < rows && word)
                *reinterpret_cast<uint32_t*>(o + e) = w[i];
        }
    }
}

// Staged rows (32 of 128 bytes, in the stores' swizzle) that bulk stores cannot
// address, to `at` + first + r ld: `rows` rows of `left` elements or fewer. A
// function of its own: its code stays out of the way of the others'.
static __device__ __noinline__ void store_rows(uint32_t sb, void* at, long long first, long long ld, int kind, int rows,
                                               int left, bool add)
{
    const int lane = threadIdx.x & 31;
    if (kind == 0) {
        float* o = static_cast<float*>(at) + first + lane;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 8, o += 8 * ld) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = __uint_as_float(ld_shared_u32(sb + (r0 + i) * 128 + ((((lane >> 2) ^ i) << 4) | ((lane & 3) << 2))));
                if (add && r0 + i < rows && lane < left)
                    v[i] += o[i * ld];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < rows && lane < left)
                    o[i * ld] = v[i];
        }
        return;
    }
    uint16_t* o = static_cast<uint16_t*>(at) + first;
    const int n = min(64, left), odd = static_cast<int>(reinterpret_cast<uintptr_t>(o) >> 1 & 1);
    // A lane a row: the first element of rows that start between two words, and the last where it is not in a word.
    if (lane < rows && n > 0) {
        const int mine = (odd + (static_cast<int>(ld) & 1) * lane) & 1;
        auto element = [&](int c) {
            const uint32_t w = ld_shared_u32(sb + lane * 128 + (((c >> 3) ^ (lane & 7)) << 4) + ((c & 6) << 1));
            return static_cast<uint16_t>(c & 1 ? w >> 16 : w);
        };
        const uint16_t first_one = element(0), last_one = element(n - 1);
        if (mine)
            o[lane * ld] = first_one;
        if ((n ^ mine) & 1)
            o[lane * ld + n - 1] = last_one;
    }
    if (ld & 1) {
        store_words<false, 2>(sb, o, ld, odd, rows, n);
        store_words<true, 2>(sb, o, ld, 1 - odd, rows, n);
    } else if (odd) {
        store_words<true, 1>(sb, o, ld, 0, rows, n);
    } else {
        store_words<false, 1>(sb, o, ld, 0, rows, n);
    }
}

// NaN in `rows` rows and `cols` columns of out[i] from (row0, col0) on, where they are in the output.
static __device__ __noinline__ void store_nan(const TileArgs& a, int i, int row0, int rows, int col0, int cols)
{
    for (int r = 0; r < min(rows, a.rows - row0); ++r)  // (row0 + rows may be 2^31)
        for (int c = threadIdx.x & 31; c < min(cols, a.cols - col0); c += 32) {
            const long long at = static_cast<long long>(row0 + r) * a.ld[i] + col0 + c;
            if (a.out_kind == 0)
                static_cast<uint32_t*>(a.out[i])[at] = 0x7FFFFFFFu;
            else
                static_cast<uint16_t*>(a.out[i])[at] = 0x7FFFu;  // a NaN of bf16 as of fp16
        }
}

struct Tile {
    int tp, tq, z;
};

// Tile t in groups of `group` tile rows, rows fastest inside a group: CTAs that
// run together share a few rows of the first operand and a few of the second.
__device__ __forceinline__ Tile tile_of(int t, const TileArgs& a)
{
    Tile w;
    const int per_z = a.tiles_p * a.tiles_q;
    w.z = t / per_z;
    t -= w.z * per_z;
    const int per = a.group * a.tiles_q;
    const int g = t / per, r = t - g * per, first = g * a.group;
    const int gs = min(a.group, a.tiles_p - first);
    w.tp = first + r % gs;
    w.tq = r / gs;
    return w;
}

// The producer's or the MMA warp's end after a wait that gave up: all that is left
// of the kernel for it, so that the loops above need no way out (with one, the
// compiler takes what follows a wait for code of single lanes, 40% slower).
template <class T>
static __device__ __noinline__ void end_warp(uint32_t tmem_base, int csize, int beside)
{
    __syncwarp();
    if (T::SPLIT && csize > 1) {
        for (int i = 0; i < 2; ++i) {
            __syncthreads();
            cluster_sync();
        }
    }
    wait_again();
    if (beside)
        wait_for_earlier();
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (T::CG == 2)
        cluster_sync();
    if (threadIdx.x >> 5 == 1) {
        tc_fence_after();
        tmem_dealloc<T::CG>(tmem_base, T::TMEM_COLS);
    }
    asm volatile("exit;");
}

template <class T>
__device__ __forceinline__ void tile_kernel(const TileMaps& maps, const ScaleMaps* scales, const TileArgs& args)
{
    extern __shared__ uint8_t smem_raw[];
    // (From one lane: the compiler then knows it to be the same in all, and keeps what the producer and the MMA warp
    // compute in uniform registers, as their instructions want it. With a lane's own values a stage cost that warp some
    // 1000 cycles, twice what the products of a 4-bit stage take.)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    const uint32_t sP = base, sQ = sP + T::STAGES * T::NP * T::P_BYTES, sS = sQ + T::STAGES * T::Q_BYTES;
    const uint32_t epi = base + T::STAGES * T::STAGE_BYTES;
    const uint32_t bars = epi + T::EPI_BYTES;
    uint8_t* const gbars = gbase + T::STAGES * T::STAGE_BYTES + T::EPI_BYTES;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (T::STAGES + s); };
    auto tfull_bar = [&](int a) { return bars + 8u * (2 * T::STAGES + a); };
    auto tempty_bar = [&](int a) { return bars + 8u * (2 * T::STAGES + 2 + a); };
    const uint32_t tmem_ready_bar = bars + 8u * (2 * T::STAGES + 4);
    auto load_bar = [&](int w) { return bars + 8u * (2 * T::STAGES + 5 + w); };  // kGrad: an epilogue warp's dh
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbars + 8 * (2 * T::STAGES + 13));
    const uint32_t abort_at = bars + 8u * (2 * T::STAGES + 13) + 4;
    static_assert(8 * (2 * T::STAGES + 14) <= T::BAR_BYTES, "barrier area");

    const uint32_t rank = T::CG == 2 || T::SPLIT ? cluster_ctarank() : 0u;
    const bool leader = T::SPLIT || rank == 0;  // of the MMA's CTA pair

    if (warp == 0) {
        if (lane < T::STAGES) {
            mbar_init(full_bar(lane), 1);
            mbar_init(empty_bar(lane), 1);
        } else if (lane < T::STAGES + 2) {
            mbar_init(tfull_bar(lane - T::STAGES), 1);
            mbar_init(tempty_bar(lane - T::STAGES), T::EPI_WARPS * T::CG);
        } else if (lane == T::STAGES + 2) {
            mbar_init(tmem_ready_bar, 1);
            st_shared_u32(abort_at, 0u);
        } else if (lane >= 16 && lane < 24) {
            mbar_init(load_bar(lane - 16), 1);
        }
        fence_mbar_init();
    }
    static_assert(T::STAGES + 3 <= 16, "one lane a barrier");
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.p[0]);
        tma_prefetch_desc(&maps.q[0]);
    }
    __syncthreads();
    if constexpr (T::CG == 2)
        cluster_sync();
    // Tensor memory is taken only now: a CTA that held it while it waited could keep it from one that it waits for. With
    // that done, the next kernel of the stream may start its set-up, or, where it needs nothing of this one, its work.
    if (!args.beside)
        wait_for_earlier();
    uint32_t tmem_base = 0;
    if (warp >= 1) {
        if (warp == 1) {
            tmem_alloc<T::CG>(smem_u32(tmem_slot), T::TMEM_COLS);
            tmem_relinquish<T::CG>();
        }
        tc_fence_before();
        named_bar_sync(1, (1 + T::EPI_WARPS) * 32);
        tc_fence_after();
        tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
        if (T::CG == 2 && !leader && warp == 1 && lane == 0)
            mbar_arrive_cluster(map_to_cta(tmem_ready_bar, 0));
    }
    if (warp == 1)
        launch_dependents();
    const Waiter wc{abort_at, T::CG == 2 ? map_to_cta(abort_at, rank ^ 1u) : abort_at};
    constexpr bool kClu = T::CG == 2;

    // Persistent: tiles t0, t0 + step, ... Split: the cluster's one tile, this
    // CTA's k-blocks [kb0, kb1).
    const int tiles = args.batch * args.tiles_p * args.tiles_q;
    const int split = T::SPLIT ? max(1, (args.num_kb + args.kb_per_rank - 1) / args.kb_per_rank) : 1;  // CTAs with a share
    const int csize = T::SPLIT ? static_cast<int>(gridDim.x) / tiles : 1;
    const int t0 = T::SPLIT ? static_cast<int>(blockIdx.x) / csize : static_cast<int>(blockIdx.x) / T::CG;
    const int step = T::SPLIT ? tiles : static_cast<int>(gridDim.x) / T::CG;
    const int kb0 = T::SPLIT ? min(args.num_kb, static_cast<int>(rank) * args.kb_per_rank) : 0;
    const int kb1 = T::SPLIT ? min(args.num_kb, kb0 + args.kb_per_rank) : args.num_kb;

    auto give_up = [&] {
        end_warp<T>(tmem_base, csize, args.beside);
        __builtin_unreachable();
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const bool one = elect_one();
        int stage = 0, wave = 0;
        uint32_t phase = 0;
        const uint32_t full0 = T::CG == 2 ? map_to_cta(full_bar(0), 0) : full_bar(0);
        for (int t = t0; t < tiles; t += step, ++wave) {
            const Tile w = tile_of(t, args);
            const int p0 = w.tp * (128 * T::CG) + (T::CG == 2 ? static_cast<int>(rank) * 128 : 0);
            const int q0 = w.tq * (T::GATED && !T::SWAP ? T::BN / 2 : T::BN);
            for (int i = 0; i < kb1 - kb0; ++i) {
                // Alternate waves run through k in opposite directions: each starts on what the last left in L2.
                const int kb = !T::SPLIT && (wave & 1) ? kb1 - 1 - i : kb0 + i;
                if (!wait_for<false>(empty_bar(stage), phase ^ 1u, wc))
                    give_up();
                const int seg = kb >= args.seg_kb ? 1 : 0;
                const int zi = seg | w.z;
                const int k0 = (kb - seg * args.seg_kb) * (T::MX ? 128 : 64);  // 4-bit maps count bytes
                const uint32_t fb = full0 + 8u * stage;
                if (one) {
                    if (T::CG == 1 || leader)
                        mbar_arrive_expect_tx(full_bar(stage), T::CG * T::TX_BYTES);
                    auto load = [&](uint32_t dst, const CUtensorMap* m, int x, int y) {
                        if constexpr (T::CG == 1)
                            tma_load_2d(dst, m, fb, x, y);
                        else
                            tma_load_2d_pair(dst, m, fb, x, y);
                    };
#pragma unroll
                    for (int n = 0; n < T::NP; ++n) {
                        const CUtensorMap* m = &maps.p[T::NP == 2 ? n : zi];
                        const uint32_t dst = sP + (stage * T::NP + n) * T::P_BYTES;
                        if constexpr (T::P_MN) {
                            load(dst, m, p0, k0);
                            load(dst + 8192, m, p0 + 64, k0);
                        } else {
                            load(dst, m, k0, p0);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < T::BN_CTA / T::QBOX; ++j) {
                        // Which part of the tile's columns box j of this CTA is: gated tiles have the gate's columns
                        // first, then the other's.
                        const int col = static_cast<int>(rank) * (T::CG == 2 ? T::BN_CTA : 0) + j * T::QBOX;
                        const int second = T::GATED && !T::SWAP && col >= T::BN / 2 ? 1 : 0;
                        const CUtensorMap* m = &maps.q[T::GATED ? second : zi];
                        const int q = q0 + col - second * (T::BN / 2);
                        const uint32_t dst = sQ + stage * T::Q_BYTES + j * (T::QBOX * 128);
                        if constexpr (T::Q_MN)
                            load(dst, m, q, k0);
                        else
                            load(dst, m, k0, q);
                    }
                    if constexpr (T::MX) {
                        const uint32_t dst = sS + stage * T::SF_BYTES;
#pragma unroll
                        for (int n = 0; n < T::NP; ++n)
                            load(dst + n * 1024, &scales->p[n], 0, (p0 >> 7) * args.sf_rows_p + kb * 2);
#pragma unroll
                        for (int j = 0; j < T::NQT; ++j) {
                            const int second = T::GATED && !T::SWAP && j * 128 >= T::BN / 2 ? 1 : 0;
                            const int q = q0 + j * 128 - second * (T::BN / 2);
                            load(dst + (T::NP + j) * 1024, &scales->q[T::GATED ? second : 0], 0,
                                 (q >> 7) * args.sf_rows_q + kb * 2);
                        }
                    }
                }
                __syncwarp();
                if (++stage == T::STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // Until every stage filled above has been read.
        for (int i = 0; i < T::STAGES; ++i) {
            if (!wait_for<false>(empty_bar(stage), phase ^ 1u, wc))
                give_up();
            if (++stage == T::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------------------------------- MMA
        if (leader) {
            const bool one = elect_one();
            int stage = 0, acc = 0;
            uint32_t acc_phase = 0;
            if constexpr (T::CG == 2) {
                if (!wait_for<true>(tmem_ready_bar, 0, wc))
                    give_up();
            }
            // The scales of a stage go to tensor memory (to columns of that stage's own) before the products of the stage
            // before it, so that no product waits for them: two words of each 128 rows of the first operand(s), then for
            // each word all row tiles of the second.
            const int per_tile = kb1 - kb0;
            const int mine = per_tile > 0 && t0 < tiles ? ((tiles - t0 + step - 1) / step) * per_tile : 0;
            int next = 0, next_stage = 0;  // the first block whose data has not been waited for, and its stage
            uint32_t next_phase = 0;
            auto arrive = [&] {
                if (!wait_for<false>(full_bar(next_stage), next_phase, wc))
                    give_up();
                tc_fence_after();
                if constexpr (T::MX) {
                    const uint32_t src = sS + next_stage * T::SF_BYTES;
                    const uint64_t sd = sdesc(src, 16, 128, 0);  // unswizzled, 8-row groups 128 bytes apart
                    const uint32_t sf0 = tmem_base + T::ACCS * T::ACC_COLS + next_stage * T::SF_COLS;
                    if (one) {
#pragma unroll
                        for (int wd = 0; wd < 2; ++wd) {
#pragma unroll
                            for (int n = 0; n < T::NP; ++n)
                                tmem_cp_scales<T::CG>(sf0 + n * 8 + wd * 4, sd + n * 64 + wd * 32);
#pragma unroll
                            for (int j = 0; j < T::NQT; ++j)
                                tmem_cp_scales<T::CG>(sf0 + T::NP * 8 + wd * 4 * T::NQT + j * 4,
                                                      sd + (T::NP + j) * 64 + wd * 32);
                        }
                    }
                    __syncwarp();
                }
                ++next;
                if (++next_stage == T::STAGES) {
                    next_stage = 0;
                    next_phase ^= 1u;
                }
            };
            const uint64_t adesc = T::P_MN ? sdesc(sP, 8192, 1024, kLayoutSW128) : sdesc(sP, 16, 1024, kLayoutSW128);
            const uint64_t bdesc = T::Q_MN ? sdesc(sQ, 8192, 1024, kLayoutSW128) : sdesc(sQ, 16, 1024, kLayoutSW128);
            int wave = 0, done = 0;
            while (done < mine) {
                if (!wait_for<kClu>(tempty_bar(acc), acc_phase ^ 1u, wc))
                    give_up();
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * T::ACC_COLS);
                for (int i = 0; i < per_tile; ++i, ++done) {
                    const int kb = !T::SPLIT && (wave & 1) ? kb1 - 1 - i : kb0 + i;
                    while (next < mine && next <= done + (T::MX ? 1 : 0))
                        arrive();
                    // (Start addresses are the descriptors' low bits, in units of 16 bytes.)
                    const uint64_t bd0 = bdesc + static_cast<uint32_t>(stage * (T::Q_BYTES / 16));
                    const uint64_t ad0 = adesc + static_cast<uint32_t>(stage * (T::NP * T::P_BYTES / 16));
                    const uint32_t sf0 = tmem_base + T::ACCS * T::ACC_COLS + stage * T::SF_COLS;
                    const int steps = T::MX && kb == args.num_kb - 1 ? args.tail_steps : 4;
                    if (one) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            if (T::MX && ks >= steps)
                                break;
                            const uint64_t bd = bd0 + ks * (T::Q_MN ? 128 : 2);
                            const uint32_t go = (i != 0 || ks != 0) ? 1u : 0u;
#pragma unroll
                            for (int n = 0; n < T::NP; ++n) {
                                const uint64_t ad = ad0 + n * (T::P_BYTES / 16) + ks * (T::P_MN ? 128 : 2);
                                if constexpr (T::MX)
                                    mma_mxf4<T::CG>(d + n * T::BN, ad, bd, args.idesc | ((ks & 1) ? kScaleIdUpper : 0u),
                                                    sf0 + n * 8 + (ks >> 1) * 4,
                                                    sf0 + T::NP * 8 + (ks >> 1) * 4 * T::NQT, go);
                                else
                                    mma_ss<T::CG, false>(d + n * T::BN, ad, bd, args.idesc, go);
                            }
                        }
                        if constexpr (T::CG == 1)
                            mma_commit(empty_bar(stage));
                        else
                            mma_commit_pair(empty_bar(stage), 0x3);
                        if (i == per_tile - 1) {
                            if constexpr (T::CG == 1)
                                mma_commit(tfull_bar(acc));
                            else
                                mma_commit_pair(tfull_bar(acc), 0x3);
                        }
                    }
                    __syncwarp();
                    if (++stage == T::STAGES)
                        stage = 0;
                }
                ++wave;
                if (++acc == T::ACCS) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
        }
        __syncwarp();
    }

    // -------------------------------------------------------------- epilogue
    const int ew = warp - 2, sub = warp & 3, half = ew >> 2;
    bool ok = true;  // false: a wait gave up, and the outputs are NaN from then on
    uint32_t acc_cols = 0;  // this tile's accumulator, at this warp's lanes
    // Adds the other CTAs' sums of a split tile, in rank order, to this one's: 4 n4 columns of row sub * 32 + lane, which
    // are group `colgroup` of the `groups` of a chunk.
    auto add_parts = [&](uint32_t* r, int n4, int chunk, int colgroup, int groups) {
        if constexpr (T::SPLIT) {
            const int per = (T::NCHUNK + split - 1) / split;  // chunks a CTA may own
            for (int s = 0; s < split - 1; ++s) {
                const uint32_t src = base + static_cast<uint32_t>((s * per + chunk / split) * T::PART_BYTES) +
                                     static_cast<uint32_t>(colgroup * (T::PART_BYTES / groups) + (sub * 32 + lane) * 16);
#pragma unroll
                for (int q = 0; q < n4; ++q) {
                    float a, b, c, d;
                    ld_shared_v4(src + q * 2048, a, b, c, d);
                    r[4 * q] = __float_as_uint(__uint_as_float(r[4 * q]) + a);
                    r[4 * q + 1] = __float_as_uint(__uint_as_float(r[4 * q + 1]) + b);
                    r[4 * q + 2] = __float_as_uint(__uint_as_float(r[4 * q + 2]) + c);
                    r[4 * q + 3] = __float_as_uint(__uint_as_float(r[4 * q + 3]) + d);
                }
            }
        }
    };
    auto own = [&](int chunk) { return !T::SPLIT || chunk % split == static_cast<int>(rank); };

    if constexpr (T::SPLIT) {
        // All CTAs' products are done (their rings are free), then every CTA sends the chunks that others own to these.
        if (warp >= 2) {
            if (kb1 > kb0)
                ok = wait_for<false>(tfull_bar(0), 0, wc);
            tc_fence_after();
            acc_cols = tmem_base + (static_cast<uint32_t>(sub * 32) << 16);
        }
        if (csize > 1) {
            __syncthreads();
            cluster_sync();
            if (warp >= 2 && kb1 > kb0) {
                const int per = (T::NCHUNK + split - 1) / split;
                for (int c = half; c < T::NCHUNK; c += 2) {
                    if (own(c))
                        continue;
                    const int to = c % split;
                    const int slot = static_cast<int>(rank) < to ? static_cast<int>(rank) : static_cast<int>(rank) - 1;
                    const uint32_t dst0 = map_to_cta(base, static_cast<uint32_t>(to)) +
                                          static_cast<uint32_t>((slot * per + c / split) * T::PART_BYTES) +
                                          static_cast<uint32_t>((sub * 32 + lane) * 16);
                    constexpr int GC = T::SWAP ? 16 : 32, GROUPS = T::CHUNK_ACC / GC;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        // Gated chunks: the gate's columns, then the other's.
                        const int col = T::GATED ? (g < GROUPS / 2 ? c * T::CHUNK + g * GC
                                                                   : (T::SWAP ? T::BN : T::BN / 2) + c * T::CHUNK +
                                                                         (g - GROUPS / 2) * GC)
                                                 : c * T::CHUNK + g * GC;
                        uint32_t r[GC];
                        if constexpr (GC == 16)
                            tmem_ld_32x32b_x16(acc_cols + col, r);
                        else
                            tmem_ld_32x32b_x32(acc_cols + col, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < GC / 4; ++q)
                            st_cluster_v4(dst0 + g * (T::PART_BYTES / GROUPS) + q * 2048, ok ? r[4 * q] : 0x7FFFFFFFu,
                                          ok ? r[4 * q + 1] : 0x7FFFFFFFu, ok ? r[4 * q + 2] : 0x7FFFFFFFu,
                                          ok ? r[4 * q + 3] : 0x7FFFFFFFu);
                    }
                }
            }
            __syncthreads();
            cluster_sync();
        }
    }

    if (warp >= 2) {
        const uint32_t sb = epi + ew * 4096;
        const uint32_t tempty0 = T::CG == 2 ? map_to_cta(tempty_bar(0), 0) : tempty_bar(0);
        int acc = 0;
        uint32_t acc_phase = 0, load_phase = 0;
        const int kind = args.out_kind, activation = args.activation;
        const float alpha = args.alpha;

        // Hands the staged 32 rows x 128 bytes (in the stores' swizzle) to out[i]: rows row0 .., columns col0 ...
        auto put = [&](int i, int row0, int col0) {
            fence_proxy_async_smem();
            __syncwarp();
            // (A box that reaches past the last column overwrites the rest of that 16-byte piece with zeros.)
            if (((args.tma_out >> i) & 1) && (args.cols - col0 >= (kind == 0 ? 32 : 64) || ((args.tma_edge >> i) & 1))) {
                if (lane == 0 && row0 < args.rows && col0 < args.cols) {
                    if (T::EPI == kStore && args.add)
                        tma_add_2d(&maps.o[i], sb, col0, row0);
                    else
                        tma_store_2d(&maps.o[i], sb, col0, row0);
                    bulk_commit();
                }
                return;
            }
            store_rows(sb, args.out[i], static_cast<long long>(row0) * args.ld[i] + col0, args.ld[i], kind,
                       min(32, args.rows - row0), args.cols - col0, T::EPI == kStore && args.add);
            __syncwarp();
        };
        // The staging buffer is free: the last store has read it.
        auto take = [&] {
            if (lane == 0)
                bulk_wait_read<0>();
            __syncwarp();
        };
        const uint32_t my_row = sb + static_cast<uint32_t>(lane * 128);
        auto piece = [&](int q) { return my_row + static_cast<uint32_t>((q ^ (lane & 7)) << 4); };

        int t = t0;
        for (; t < tiles; t += step) {
            const Tile w = tile_of(t, args);
            const int row0 = w.tp * (128 * T::CG) + (T::CG == 2 ? static_cast<int>(rank) * 128 : 0) + sub * 32;
            const int col0 = w.tq * T::OUT_COLS;
            if constexpr (!T::SPLIT) {
                if constexpr (T::EPI == kGrad) {
                    // dh comes into the staging buffer while the products run.
                    take();
                    if (ok && lane == 0 && half < T::NCHUNK && row0 < args.rows && col0 + half * 64 < args.cols) {
                        mbar_arrive_expect_tx(load_bar(ew), 4096);
                        tma_load_2d(sb, &maps.o[2], load_bar(ew), col0 + half * 64, row0);
                    }
                }
                if (ok)
                    ok = wait_for<false>(tfull_bar(acc), acc_phase, wc);
                tc_fence_after();
                acc_cols = tmem_base + (static_cast<uint32_t>(sub * 32) << 16) + static_cast<uint32_t>(acc * T::ACC_COLS);
            }
            // One group of accumulator columns, scaled.
            auto fetch32 = [&](float (&v)[32], int col, int chunk, int group) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(acc_cols + col, r);
                tmem_wait_ld();
                add_parts(r, 8, chunk, group, T::CHUNK_ACC / 32);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = alpha * __uint_as_float(r[j]);
            };
            auto release = [&] {
                if constexpr (!T::SPLIT) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (T::CG == 1)
                            mbar_arrive(tempty0 + 8u * acc);
                        else
                            mbar_arrive_cluster(tempty0 + 8u * acc);
                    }
                }
            };

            auto stage16 = [&](const float (&x)[32], int at) {  // 32 values of this row as 16-bit columns from `at` on
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4u(piece(at / 8 + q), pack2(x[8 * q], x[8 * q + 1], kind), pack2(x[8 * q + 2], x[8 * q + 3], kind),
                                  pack2(x[8 * q + 4], x[8 * q + 5], kind), pack2(x[8 * q + 6], x[8 * q + 7], kind));
            };
            if (!ok)
                break;
            if constexpr (T::DRAIN) {
                // This warp's columns go to registers at once, and the accumulator back to the MMA warp (of one accumulator
                // the next tile's products begin now). Half the tile's columns a warp: 64 of each factor of a gated tile,
                // else two chunks of 64.
                float v[4][32];
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    tmem_ld_32x32b_x32(acc_cols + (T::GATED ? (g >> 1) * (T::BN / 2) + half * 64 + (g & 1) * 32
                                                            : half * 128 + g * 32),
                                       reinterpret_cast<uint32_t(&)[32]>(v[g]));
                tmem_wait_ld();
                release();
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[g][j] = alpha * v[g][j];
                constexpr int GROUPS = T::GATED ? 2 : 4;
                static_assert(GROUPS * 32 == T::RUN, "the columns that are NaN where a wait gives up");
                const int first = col0 + half * T::RUN;
                if constexpr (T::GATED) {
                    if (!T::MX && args.keep) {
                        take();
                        stage16(v[0], 0);
                        stage16(v[1], 32);
                        put(1, row0, first);
                        take();
                        stage16(v[2], 0);
                        stage16(v[3], 32);
                        put(2, row0, first);
                    }
                    gate<T>(v[0], v[2], activation, kind);
                    gate<T>(v[1], v[3], activation, kind);
                }
                if (T::MX && kind == 0) {  // (fp32 outputs: of 4-bit operands only)
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        take();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_v4(piece(q), v[g][4 * q], v[g][4 * q + 1], v[g][4 * q + 2], v[g][4 * q + 3]);
                        put(0, row0, first + g * 32);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < GROUPS; g += 2) {
                        take();
                        stage16(v[g], 0);
                        stage16(v[g + 1], 32);
                        put(0, row0, first + g * 32);
                    }
                }
            } else if constexpr (T::SWAP) {
                // This lane's accumulator row is output column f, its columns are tokens.
                const int f = row0 + lane;
                for (int c = half; c < T::NCHUNK; c += 2) {
                    if (!own(c))
                        continue;
                    const int tok0 = col0 + c * 16;
                    uint32_t r[16];
                    float g[16], u[16];
                    auto take16 = [&](float (&v)[16], int col, int group) {
                        tmem_ld_32x32b_x16(acc_cols + col, r);
                        tmem_wait_ld();
                        add_parts(r, 4, c, group, T::CHUNK_ACC / 16);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            v[j] = alpha * __uint_as_float(r[j]);
                    };
                    take16(g, c * 16, 0);
                    if constexpr (T::GATED)
                        take16(u, T::BN + c * 16, 1);
                    const int n = f < args.cols ? args.rows - tok0 : 0;
                    if constexpr (T::GATED) {
                        if (args.keep) {
                            store_column(args.out[1], kind, tok0 * args.ld[1] + f, args.ld[1], n, g);
                            store_column(args.out[2], kind, tok0 * args.ld[2] + f, args.ld[2], n, u);
                        }
                        gate<T>(g, u, activation, kind);
                    }
                    store_column(args.out[0], kind, tok0 * args.ld[0] + f, args.ld[0], n, g);
                }
            } else if constexpr (T::SPLIT) {
                // 32 output columns at a time, dealt to the CTAs and to both halves of the warps: with 64, half of the warps
                // of half of the CTAs added up a gated tile's sums. Rows on 16 bytes go straight out of the registers.
                auto out32 = [&](int i, const float (&x)[32], int cc) {
                    if (kind == 0) {
                        take();
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            st_shared_v4(piece(q), x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                        put(i, row0, cc);
                        return;
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        p[q] = pack2(x[2 * q], x[2 * q + 1], kind);
                    if (((args.tma_out >> i) & 1) && args.cols - cc >= 32) {
                        if (row0 + lane < args.rows) {
                            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out[i]) +
                                                                static_cast<long long>(row0 + lane) * args.ld[i] + cc);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                o[q] = make_uint4(p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
                        }
                        return;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        st_shared_v4u(piece(q), p[4 * q], p[4 * q + 1], p[4 * q + 2], p[4 * q + 3]);
                    __syncwarp();
                    store_rows(sb, args.out[i], static_cast<long long>(row0) * args.ld[i] + cc, args.ld[i], kind,
                               min(32, args.rows - row0), min(32, args.cols - cc), false);
                    __syncwarp();
                };
#pragma unroll 1
                for (int c = half; c < T::NCHUNK; c += 2) {
                    if (!own(c))
                        continue;
                    const int cc = col0 + c * 32;
                    if constexpr (T::EPI == kGrad) {
                        fence_proxy_async_smem();
                        take();
                        if (row0 < args.rows && cc < args.cols) {
                            if (lane == 0) {
                                mbar_arrive_expect_tx(load_bar(ew), 4096);
                                tma_load_2d(sb, &maps.o[2], load_bar(ew), cc, row0);
                            }
                            ok = wait_for<false>(load_bar(ew), load_phase, wc);
                            load_phase ^= 1u;
                        }
                        if (!ok)
                            break;
                    }
                    float v[32];
                    fetch32(v, c * 32, c, 0);
                    if constexpr (!T::GATED) {
                        out32(w.z, v, cc);
                    } else {
                        float u[32];
                        fetch32(u, T::BN / 2 + c * 32, c, 1);
                        if constexpr (T::EPI == kGated) {
                            if (args.keep) {
                                out32(1, v, cc);
                                out32(2, u, cc);
                            }
                            gate<T>(v, u, activation, kind);
                            out32(0, v, cc);
                        } else {
                            uint32_t hw[16];  // this row's 32 values of dh (of the 64 that a box brings)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                ld_shared_v4u(piece(q), hw[4 * q], hw[4 * q + 1], hw[4 * q + 2], hw[4 * q + 3]);
                            slope(v, u, hw, kind, activation);
                            out32(0, v, cc);
                            out32(1, u, cc);
                        }
                    }
                }
                if (!ok)
                    break;
            } else if constexpr (T::EPI == kStore) {
#pragma unroll 1
                for (int c = half; c < T::NCHUNK; c += 2) {
                    if (kind == 0) {
#pragma unroll 1
                        for (int g = 0; g < 2; ++g) {
                            float v[32];
                            fetch32(v, c * 64 + g * 32, c, g);
                            if (c + 2 >= T::NCHUNK && g == 1)
                                release();
                            take();
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                st_shared_v4(piece(q), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                            put(w.z, row0, col0 + c * 64 + g * 32);
                        }
                    } else {
                        take();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float v[32];
                            fetch32(v, c * 64 + g * 32, c, g);
                            if (c + 2 >= T::NCHUNK && g == 1)
                                release();
                            stage16(v, g * 32);
                        }
                        put(w.z, row0, col0 + c * 64);
                    }
                }
            } else {
                static_assert(T::EPI == kGrad && T::NCHUNK == 2, "a chunk a warp");
                const int c = half, cc = col0 + c * 64;
                uint32_t hw[32];  // this row's 64 values of dh, then of du
                if (row0 < args.rows && cc < args.cols) {
                    ok = wait_for<false>(load_bar(ew), load_phase, wc);
                    load_phase ^= 1u;
                }
                if (!ok)
                    break;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    ld_shared_v4u(piece(q), hw[4 * q], hw[4 * q + 1], hw[4 * q + 2], hw[4 * q + 3]);
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float v[32], u[32];
                    fetch32(v, c * 64 + g * 32, c, g);
                    fetch32(u, T::BN / 2 + c * 64 + g * 32, c, 2 + g);
                    if (g == 1)
                        release();
                    uint32_t d[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        d[j] = hw[g * 16 + j];
                    slope(v, u, d, kind, activation);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        hw[g * 16 + j] = pack2(u[2 * j], u[2 * j + 1], kind);
                    stage16(v, g * 32);
                }
                put(0, row0, cc);
                take();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    st_shared_v4u(piece(q), hw[4 * q], hw[4 * q + 1], hw[4 * q + 2], hw[4 * q + 3]);
                put(1, row0, cc);
            }
            if (++acc == T::ACCS) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        for (; t < tiles; t += step) {  // a wait gave up: this warp's outputs of the tiles that are left
            const Tile w = tile_of(t, args);
            const int row0 = w.tp * (128 * T::CG) + (T::CG == 2 ? static_cast<int>(rank) * 128 : 0) + sub * 32;
            const int outs = T::EPI == kGrad ? 2 : T::EPI == kGated && args.keep ? 3 : 1;
            for (int o = 0; o < outs; ++o)
                for (int c = half; c < T::RUNS; c += 2) {
                    if (!own(c))
                        continue;
                    const int col = w.tq * T::OUT_COLS + c * T::RUN;
                    if (T::SWAP)
                        store_nan(args, o, col, T::RUN, row0, 32);
                    else
                        store_nan(args, T::EPI == kStore ? w.z : o, row0, 32, col, T::RUN);
                }
        }
        if (!T::SWAP && lane == 0) {
            bulk_wait<0>();
            fence_proxy_async_global();
        }
        __syncwarp();
    }

    if (__any_sync(0xffffffffu, wc.aborted()))
        wait_again();
    if (args.beside)
        wait_for_earlier();  // this kernel's end is the end of the one before, too
    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if constexpr (T::CG == 2)
        cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<T::CG>(tmem_base, T::TMEM_COLS);
    }
}

template <class T>
__global__ void __launch_bounds__(T::THREADS, T::SWAP && T::BN <= 32 ? 2 : 1)
    sat_ffn_tile_kernel(const __grid_constant__ TileMaps maps, const TileArgs args)
{
    tile_kernel<T>(maps, nullptr, args);
}

template <class T>
__global__ void __launch_bounds__(T::THREADS, T::SWAP && T::BN <= 32 ? 2 : 1)
    sat_ffn_scaled_tile_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ ScaleMaps scales, const TileArgs args)
{
    tile_kernel<T>(maps, &scales, args);
}

template <class T>
const void* tile_function()
{
    if constexpr (T::MX)
        return reinterpret_cast<const void*>(sat_ffn_scaled_tile_kernel<T>);
    else
        return reinterpret_cast<const void*>(sat_ffn_tile_kernel<T>);
}

// The kernel's shared memory is allowed on the current device (asked for once for each).
template <class T>
cudaError_t allow_memory(int* device)
{
    const void* fn = tile_function<T>();
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    *device = dev;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

// The CTAs of a cluster are of one GPC, and the GPCs' sizes differ from chip to chip: 152 SMs held 76, 46, 36, 28, 23, 15 and
// 15 clusters of 2 to 8 CTAs of an SM each. A cluster too many runs after the others: 20.8 us instead of 14.0 (96 x 4096 x 1024).
template <class T>
cudaError_t clusters_at_once(int cluster, int* clusters)
{
    static std::atomic<int> known[64][9];
    int dev = 0;
    cudaError_t e = allow_memory<T>(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && (*clusters = known[dev][cluster].load(std::memory_order_relaxed)) > 0)
        return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(T::THREADS);
    cfg.dynamicSmemBytes = T::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, tile_function<T>(), &cfg);
    if (e == cudaSuccess && dev < 64)
        known[dev][cluster].store(*clusters, std::memory_order_relaxed);
    return e;
}

template <class T>
cudaError_t launch_tiles(const TileMaps& maps, const ScaleMaps* scales, const TileArgs& args, int grid, int cluster,
                         cudaStream_t stream)
{
    int dev = 0;
    const cudaError_t e = allow_memory<T>(&dev);
    if (e != cudaSuccess)
        return e;
    if constexpr (T::MX)
        return launch_early(sat_ffn_scaled_tile_kernel<T>, static_cast<unsigned>(grid), T::THREADS, T::SMEM_BYTES,
                            static_cast<unsigned>(cluster), stream, maps, *scales, args);
    else
        return launch_early(sat_ffn_tile_kernel<T>, static_cast<unsigned>(grid), T::THREADS, T::SMEM_BYTES,
                            static_cast<unsigned>(cluster), stream, maps, args);
}

template <class T>
constexpr Variant variant()
{
    return Variant{T::MX, T::EPI, T::CG, T::BN, T::P_MN, T::Q_MN, T::SWAP, !T::SPLIT,
                   T::STAGES * T::STAGE_BYTES, T::NCHUNK, T::PART_BYTES, &launch_tiles<T>, &clusters_at_once<T>};
}

}  // namespace ffn
}  // namespace sat
