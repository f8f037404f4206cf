// What the row operators of language models share: element types, loads and
// stores of eight elements, reductions over a CTA, and checks of arguments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"
#include "registry.h"
#include "rowops.h"

namespace sat {
namespace rows {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v)
{
    if constexpr (std::is_same_v<T, float>)
        return v;
    else if constexpr (std::is_same_v<T, __half>)
        return __float2half_rn(v);
    else
        return __float2bfloat16_rn(v);
}

// Eight consecutive elements as they lie in memory, 16 or 32 bytes, moved by
// one instruction (256-bit global loads and stores for fp32). The address is
// aligned to the eight elements.
template <typename T>
struct Pack {
    uint32_t w[2 * sizeof(T)];
};

template <typename T>
__device__ __forceinline__ Pack<T> load_pack(const T* p)
{
    Pack<T> v;
    if constexpr (sizeof(T) == 4)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
                       "=r"(v.w[6]), "=r"(v.w[7])
                     : "l"(p));
    else
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3])
                     : "l"(p));
    return v;
}

template <typename T>
__device__ __forceinline__ void store_pack(T* p, const Pack<T>& v)
{
    if constexpr (sizeof(T) == 4)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]),
                     "r"(v.w[2]), "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                     : "memory");
    else
        asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]),
                     "r"(v.w[3])
                     : "memory");
}

// The two 16-bit elements of a word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w)
{
    if constexpr (std::is_same_v<T, __half>)
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T>
__device__ __forceinline__ void unpack(const Pack<T>& v, float (&out)[8])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            out[e] = __uint_as_float(v.w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<T>(v.w[e]);
            out[2 * e] = f.x;
            out[2 * e + 1] = f.y;
        }
    }
}

template <typename T>
__device__ __forceinline__ Pack<T> pack(const float (&in)[8])
{
    Pack<T> v;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v.w[e] = __float_as_uint(in[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (std::is_same_v<T, __half>) {
                const __half2 h = __floats2half2_rn(in[2 * e], in[2 * e + 1]);
                v.w[e] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(in[2 * e], in[2 * e + 1]);
                v.w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    return v;
}

// Sixteen bytes as they lie in memory, and their elements.
template <typename T>
constexpr int kPer16 = 16 / sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& w, float (&out)[kPer16<T>])
{
    if constexpr (sizeof(T) == 4) {
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            out[e] = __uint_as_float(words[e]);
    } else {
        Pack<T> v = {{w.x, w.y, w.z, w.w}};
        unpack(v, out);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&in)[kPer16<T>])
{
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(in[0]), __float_as_uint(in[1]), __float_as_uint(in[2]), __float_as_uint(in[3]));
    } else {
        const Pack<T> v = pack<T>(in);
        return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
}

// A row as packs of 16 bytes on their boundaries in memory: pack i starts with
// element i N - shift, and those from `inside` to `end` lie wholly in the row.
template <typename T>
struct Packs {
    static constexpr int N = kPer16<T>;
    const T* row;
    int vocab, shift, count, inside, end;

    __device__ __forceinline__ Packs(const T* r, int v) : row(r), vocab(v)
    {
        shift = static_cast<int>((reinterpret_cast<uint64_t>(r) & 15) / sizeof(T));
        count = (v + shift + N - 1) / N;
        inside = shift ? 1 : 0;
        end = max((v + shift) / N, inside);
    }
    __device__ __forceinline__ int element(int i) const { return i * N - shift; }
    __device__ __forceinline__ uint4 load(int i) const { return *reinterpret_cast<const uint4*>(row + element(i)); }
};

// Sums of N values over the NT threads that share a row, returned to each of
// them, in a fixed order: lanes by shuffles, then (NT > 32) warps through
// `scratch`, 2 x N x NT / 32 floats. Consecutive reductions alternate between
// its halves, so one barrier each suffices: a half is rewritten two
// reductions later, after a barrier that every thread passed after reading it.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* scratch, int& turn)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (NT > 32) {
        constexpr int W = NT / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float* half = scratch + turn * (N * W);
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i)
                half[i * W + warp] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = lane < W ? half[i * W + lane] : 0.0f;
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if constexpr (W < 32)
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = __shfl_sync(0xffffffffu, v[i], 0);
    }
}

// 2^x, flushing what is below the smallest normal number to 0 (relative error
// about 2^-22; one instruction, where exp2f adds the care for subnormals).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x to about 2^-23, flushing subnormals.
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The scale of a softmax's exponents at temperature t, log2 e / t: finite also
// where t is below the smallest normal number, so that equal logits stay equal
// (0 times it is 0).
__device__ __forceinline__ float scale_at(float t) { return fminf(kLog2e / t, FLT_MAX); }

// Two fp32 values in one 64-bit register, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 halves(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// Sixteen bytes as pairs of fp32 values, and the largest of them (NaNs aside).
template <typename T>
constexpr int kPairs = 8 / sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& w, uint64_t (&out)[kPairs<T>])
{
    if constexpr (sizeof(T) == 4) {
        out[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
        out[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
    } else {
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<T>(words[e]);
            out[e] = pair(f.x, f.y);
        }
    }
}

template <typename T>
__device__ __forceinline__ float largest(const uint4& w)
{
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    } else {
        using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
        const T2 m = __hmax2(__hmax2(*reinterpret_cast<const T2*>(&w.x), *reinterpret_cast<const T2*>(&w.y)),
                             __hmax2(*reinterpret_cast<const T2*>(&w.z), *reinterpret_cast<const T2*>(&w.w)));
        const float2 f = unpack2<T>(*reinterpret_cast<const uint32_t*>(&m));
        return fmaxf(f.x, f.y);
    }
}

// The maximum of a softmax's values and the sum of 2^((v - max) scale) over
// them, scale being log2 e over the temperature. The difference comes first:
// it is exact where it matters, so rows far from 0 lose nothing, and it is 0
// where all values are the type's lowest, whose products overflow.
struct Softmax {
    float max, sum;

    static __device__ __forceinline__ Softmax none() { return {-INFINITY, 0.0f}; }

    __device__ __forceinline__ void add(float v, float scale)
    {
        if (v > max) {
            sum *= ex2((max - v) * scale);
            max = v;
        }
        // With nothing but -inf so far 0 is subtracted, so that 2^-inf is 0. A NaN stays in the sum.
        sum += ex2((v - (max == -INFINITY ? 0.0f : max)) * scale);
    }

    __device__ __forceinline__ void add(const Softmax& o, float scale)
    {
        const float m = fmaxf(max, o.max);
        // A side that has seen nothing but -inf keeps its sum of 0 (or NaN).
        sum = (max == m ? sum : sum * ex2((max - m) * scale)) + (o.max == m ? o.sum : o.sum * ex2((o.max - m) * scale));
        max = m;
    }
};

// Sums of 2^((v - top) scale) over packs of 16 bytes, `get(i)` for i < n: for
// each pair of elements a multiply-add, two exponentials and an addition. The
// multiply-add subtracts top scale as rounded, and what the rounding was goes
// into the sum as a factor at the end, so rows far from 0 lose nothing. That
// holds while the rounding is a small part of a binade: below 2^20 it is at most
// 2^-5. Beyond (masks of -1e9, a tiny temperature), where it may be hundreds of
// binades, and where the product overflows (the type's lowest value), the
// difference is taken first instead, one instruction more.
template <typename T, typename Get>
__device__ __forceinline__ float sum_packs(Get get, int n, float top, float scale)
{
    const float from = top == -INFINITY ? 0.0f : top;  // of nothing but -inf: 0 is subtracted, and 2^-inf is 0
    const bool plain = fabsf(from * scale) < 0x1p20f;
    const float off = plain ? -from * scale : -from;
    const uint64_t scale2 = pair(scale, scale), off2 = pair(off, off);
    uint64_t sums[2] = {0, 0};
    if (plain) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            uint64_t v[kPairs<T>];
            unpack_pairs<T>(get(i), v);
#pragma unroll
            for (int e = 0; e < kPairs<T>; ++e) {
                const float2 x = halves(fma2(v[e], scale2, off2));
                sums[e & 1] = add2(sums[e & 1], pair(ex2(x.x), ex2(x.y)));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            uint64_t v[kPairs<T>];
            unpack_pairs<T>(get(i), v);
#pragma unroll
            for (int e = 0; e < kPairs<T>; ++e) {
                const float2 x = halves(mul2(add2(v[e], off2), scale2));
                sums[e & 1] = add2(sums[e & 1], pair(ex2(x.x), ex2(x.y)));
            }
        }
    }
    const float2 s = halves(add2(sums[0], sums[1]));
    return (s.x + s.y) * (plain ? ex2(-fmaf(from, scale, off)) : 1.0f);
}

// A pack of -inf, for where a row has none.
template <typename T>
__device__ __forceinline__ uint4 nothing()
{
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same_v<T, __half> ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
}

// The softmax of a thread's packs, all of them in registers: the maximum
// first, so that no sum is rescaled.
template <typename T, int U>
__device__ __forceinline__ Softmax softmax_of(const uint4 (&w)[U], float scale)
{
    float top = largest<T>(w[0]);
#pragma unroll
    for (int u = 1; u < U; ++u)
        top = fmaxf(top, largest<T>(w[u]));
    return {top, sum_packs<T>([&](int i) { return w[i]; }, U, top, scale)};
}

// The softmax over what a warp's lanes have seen, to each of them: the largest
// maximum first, so that a lane rescales its sum once.
__device__ __forceinline__ Softmax warp_softmax(Softmax s, float scale)
{
    float m = s.max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // A lane that has seen nothing but -inf keeps its sum of 0 (or NaN).
    float sum = s.max == m ? s.sum : s.sum * ex2((s.max - m) * scale);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return {m, sum};
}

// The softmax of n shares that lie in memory, in order.
__device__ __forceinline__ Softmax sum_softmax(const Softmax* s, int stride, int n, float scale)
{
    float m = s[0].max, sum = 0.0f;
    for (int i = 1; i < n; ++i)
        m = fmaxf(m, s[i * stride].max);
    for (int i = 0; i < n; ++i)
        sum += s[i * stride].max == m ? s[i * stride].sum : s[i * stride].sum * ex2((s[i * stride].max - m) * scale);
    return {m, sum};
}

// The softmax over what the NT threads of a CTA have seen, returned to each of
// them, in a fixed order. `scratch` holds NT / 32 of them; free after a barrier.
template <int NT>
__device__ __forceinline__ Softmax cta_softmax(Softmax s, float scale, Softmax* scratch)
{
    s = warp_softmax(s, scale);
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = s;
    __syncthreads();
    return warp_softmax((threadIdx.x & 31) < NT / 32 ? scratch[threadIdx.x & 31] : Softmax::none(), scale);
}

// ---- bounded waits -----------------------------------------------------------------

// Every wait for a copy or for another CTA's sums gives up after two seconds,
// more than any launch takes. Whoever gave up has NaN for what it was to
// compute, waits for nothing more and sends, fills and releases nothing more
// (a barrier is armed again only by those who have seen its phase end). A CTA
// ends when the copies that it has started have landed, or have had that time
// again, and one of a cluster not before the others. Tests build with 0: then
// a wait gives up at its first look.
#ifndef SAT_ROWS_WAIT_NS
#define SAT_ROWS_WAIT_NS 2000000000ull
#endif
constexpr uint64_t kWaitNs = SAT_ROWS_WAIT_NS, kDrainNs = 2000000000ull;
constexpr uint64_t kSettleNs = kWaitNs ? kWaitNs : 10000000ull;

// Whether the barrier's phase of this parity ended within the limit.
template <bool kCluster, uint64_t kLimitNs = kWaitNs>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity)
{
    if constexpr (kLimitNs == 0) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
        return ok != 0;
    } else {
        uint64_t since = 0;
        for (unsigned n = 1; !mbar_try_wait<kCluster>(bar, parity); ++n)
            if (n % 32 == 0) {
                const uint64_t now = globaltimer_ns();
                if (n == 32)
                    since = now;
                else if (now - since > kLimitNs)
                    return false;
            }
        return true;
    }
}

// ---- clusters ----------------------------------------------------------------------

// Stores to shared memory of any CTA of the cluster (which must have started).
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Stores eight bytes to shared memory of any CTA of the cluster and counts them on a barrier there.
__device__ __forceinline__ void send_b64(uint32_t addr, uint64_t v, uint32_t bar)
{
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(addr), "l"(v), "r"(bar)
                 : "memory");
}

// The halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---- host: kernels' attributes -----------------------------------------------------

// Sets, once per kernel and device, how much dynamic shared memory the kernel
// may have and that its clusters may have up to 16 CTAs. Zero-initialised
// statics, safe from several threads.
struct Prepared {
    std::atomic<uint64_t> devices[2];

    cudaError_t once(const void* kernel, int smem)
    {
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess || (d < 128 && (devices[d / 64].load(std::memory_order_acquire) >> (d % 64) & 1)))
            return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && d < 128)
            devices[d / 64].fetch_or(uint64_t{1} << (d % 64), std::memory_order_release);
        return e;
    }
};

// ---- host: argument checks ------------------------------------------------------

inline bool type_ok(int t) { return t == GEMM_C_F32 || t == GEMM_C_BF16 || t == GEMM_C_F16; }
inline int type_bytes(int t) { return t == GEMM_C_F32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether all rows start on a boundary of eight elements (a matrix that is not there does).
inline bool packs(const void* p, int64_t ld, int type) { return !p || (aligned(p, 8 * type_bytes(type)) && ld % 8 == 0); }

}  // namespace rows
}  // namespace sat
