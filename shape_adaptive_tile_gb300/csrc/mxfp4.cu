// Microscaled 4-bit matrices: quantisation and its inverse (include/ffn.h).
#include <cuda_fp4.h>

#include "ffn.h"
#include "ffn_ptx.cuh"
#include "ffn_tile.h"
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 256;

struct Args {
    long long rows, width, ldv, ldc;
    int blocks;    // of 32 columns, of a row
    int groups;    // of four blocks, of a row: one word of scales
    int per_row;   // threads that take a row's columns in one go, eight each: 16 times a number of groups
    int chunks;    // goes that a row takes
    long long sets;  // sets of four rows, 32 apart in a tile of 128: their words of scales are 16 consecutive bytes
    void* values;
    uint8_t* codes;
    uint4* scales;  // by group and row within 32 of a tile
};

// What a thread does: columns 8 unit .., rows row + 32 u, scales[at].
struct Place {
    bool in;
    int unit;
    long long row, at;
};

__device__ __forceinline__ Place place(const Args& a)
{
    Place p;
    const unsigned go = blockIdx.x / a.chunks, chunk = blockIdx.x - go * a.chunks;
    const int sub = threadIdx.x / a.per_row, rows = kThreads / a.per_row;
    const long long set = static_cast<long long>(go) * rows + sub;
    p.unit = chunk * a.per_row + threadIdx.x - sub * a.per_row;
    p.in = sub < rows && set < a.sets && p.unit < a.groups * 16;
    p.row = (set >> 5) * 128 + (set & 31);
    p.at = ((set >> 5) * a.groups + (p.unit >> 4)) * 32 + (set & 31);
    return p;
}

// Eight elements of row[j ..]; past the width 0. Rows that start off 16 bytes:
// by the 16-byte pieces around them where these lie in the row, shifted into
// place (the shift is the same in all of a row's threads).
template <typename T, bool kVec>
__device__ __forceinline__ Pack<T> load8(const T* row, long long j, long long width)
{
    if (kVec && j + 8 <= width)
        return load_pack(row + j);
    Pack<T> v{};
    if constexpr (!kVec) {
        constexpr int P = 16 / sizeof(T), N = sizeof(T) == 4 ? 3 : 2;
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + j)) & 15u;
        const int back = static_cast<int>(off / sizeof(T));
        if (j >= back && j - back + N * P <= width) {
            const uint4* from = reinterpret_cast<const uint4*>(row + j - back);
            uint32_t w[4 * N + 3] = {};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint4 q = __ldg(from + i);
                w[4 * i] = q.x;
                w[4 * i + 1] = q.y;
                w[4 * i + 2] = q.z;
                w[4 * i + 3] = q.w;
            }
#pragma unroll
            for (int i = 0; i < 4 * N; ++i)
                w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 4 * N; ++i)
                w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i)
                v.w[i] = sizeof(T) == 2 && (off & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
            return v;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (j + i < width)
            reinterpret_cast<T*>(v.w)[i] = row[j + i];
    return v;
}

// The exponent field, as an fp32 number's, of the largest magnitude: 255 with an infinity or a NaN among the values.
__device__ __forceinline__ uint32_t largest_field(const Pack<float>& p)
{
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        top = max(top, p.w[k] & 0x7FFFFFFFu);
    return top >> 23;
}

template <typename T>
__device__ __forceinline__ uint32_t largest_field(const Pack<T>& p)  // 16-bit types: two values at a time
{
    uint32_t two = p.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int k = 1; k < 4; ++k)
        two = __vmaxu2(two, p.w[k] & 0x7FFF7FFFu);
    const uint16_t top = static_cast<uint16_t>(max(two & 0xFFFFu, two >> 16));
    return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&top))) >> 23;
}

// Eight columns of four rows a thread, all loads in flight at once: four
// threads a block of 32, sixteen a word of scales. The exponent field of a
// block's largest magnitude is its logarithm rounded down (bits compare as
// magnitudes do); the four rows' fields share a word, whose bytes are compared
// and exchanged together: 4 shuffles for 32 values a thread instead of 16.
// Bounded by the reads; 8192 x 8192 bf16: see the table of cases.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) sat_mxfp4_quantize_kernel(const __grid_constant__ Args a)
{
    launch_dependents();
    wait_for_earlier();
    const Place p = place(a);
    const long long j = p.unit * 8ll;
    Pack<T> in[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (p.in && p.row + 32 * u < a.rows)
            in[u] = load8<T, kVec>(static_cast<const T*>(a.values) + (p.row + 32 * u) * a.ldv, j, a.width);
        else
            in[u] = Pack<T>{};
    uint32_t fields = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        fields |= largest_field(in[u]) << (8 * u);
    fields = __vmaxu4(fields, __shfl_xor_sync(0xffffffffu, fields, 1));
    fields = __vmaxu4(fields, __shfl_xor_sync(0xffffffffu, fields, 2));
    // exponent + 127 of each row's block: two less, not below 0, and 255 for what is not finite.
    const uint32_t bytes = __vsubus4(fields, 0x02020202u) | __vcmpeq4(fields, 0xFFFFFFFFu);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t byte = bytes >> (8 * u) & 255u;
        const float by = __uint_as_float((254u - byte) << 23);  // 2^-exponent, always a normal number (of 255: not used)
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = make_float2(to_f32(reinterpret_cast<const T*>(in[u].w)[2 * k]) * by,
                                         to_f32(reinterpret_cast<const T*>(in[u].w)[2 * k + 1]) * by);
            w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * k);
        }
        if (p.in && p.row + 32 * u < a.rows && (p.unit >> 2) < a.blocks)
            *reinterpret_cast<uint32_t*>(a.codes + (p.row + 32 * u) * a.ldc + p.unit * 4) = byte == 255 ? 0u : w;
    }
    // The bytes of four blocks x four rows, each block's in one group of lanes, turned: group g gets row g's word.
    const int g = threadIdx.x >> 2 & 3;
    uint32_t other = __shfl_xor_sync(0xffffffffu, bytes, 4);
    uint32_t word = __byte_perm(bytes, other, g & 1 ? 0x3715 : 0x6240);
    other = __shfl_xor_sync(0xffffffffu, word, 8);
    word = __byte_perm(word, other, g & 2 ? 0x3276 : 0x5410);
    if (p.in && (threadIdx.x & 3) == 0)
        reinterpret_cast<uint32_t*>(a.scales + p.at)[g] = word;  // 0 for rows past the last one
}

// Eight elements a thread to row[j ..], of rows that start off 16 bytes (all of a
// warp's threads; `in`: this one has elements). A thread writes the 16-byte
// pieces that begin among its elements, the last of them with the next lane's;
// elements at the row's or the warp's ends, in no such piece, go one by one.
// (All one by one, 8192 x 8191 bf16 took 174 us instead of 36.)
template <typename T>
__device__ __forceinline__ void store_shifted(T* row, long long j, long long width, const Pack<T>& v, bool in, bool same_as_next,
                                              bool same_as_last)
{
    constexpr int P = 16 / sizeof(T), W = 2 * sizeof(T), PIECES = W / 4;
    uint32_t w[W + 4 + 3] = {};
#pragma unroll
    for (int i = 0; i < W; ++i)
        w[i] = v.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[W + i] = __shfl_down_sync(0xffffffffu, v.w[i], 1);
    if (!in)
        return;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + j)) & 15u, skip = (16u - off) & 15u;
    const int first = static_cast<int>(skip / sizeof(T));  // element that the first piece begins with
#pragma unroll
    for (int i = 0; i < W + 4; ++i)
        w[i] = skip & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < W + 4; ++i)
        w[i] = skip & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < W; ++i)
        w[i] = sizeof(T) == 2 && (skip & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    int done = first;  // elements from `first` on that pieces take
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
        const bool mine = first + (k + 1) * P <= 8;
        if (j + first + (k + 1) * P <= width && (mine || same_as_next)) {
            *reinterpret_cast<uint4*>(row + j + first + k * P) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            done = first + (k + 1) * P;
        }
    }
    const bool head = first > 0 && !(same_as_last && j + first <= width);  // no piece of the last lane's reaches in here
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if ((i < first ? head : i >= done) && j + i < width)
            row[j + i] = reinterpret_cast<const T*>(v.w)[i];
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) sat_mxfp4_dequantize_kernel(const __grid_constant__ Args a)
{
    launch_dependents();
    wait_for_earlier();
    const Place p = place(a);
    const bool in = p.in && (p.unit >> 2) < a.blocks;
    if (kVec && !in)
        return;
    const long long j = p.unit * 8ll;
    const uint4 s4 = in ? a.scales[p.at] : make_uint4(0, 0, 0, 0);
    const uint32_t words[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t codes[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        codes[u] = in && p.row + 32 * u < a.rows
                       ? *reinterpret_cast<const uint32_t*>(a.codes + (p.row + 32 * u) * a.ldc + p.unit * 4)
                       : 0u;
    // Whether the neighbouring lanes have the row's next and last eight columns.
    const int lane = threadIdx.x & 31, in_row = threadIdx.x % a.per_row;
    const bool same_as_next = lane < 31 && in_row + 1 < a.per_row, same_as_last = lane > 0 && in_row > 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const bool here = in && p.row + 32 * u < a.rows;
        const uint32_t byte = words[u] >> (8 * (p.unit / 4 % 4)) & 255u;
        // 2^(byte - 127): of byte 0 it is below the normal numbers.
        const float by = __uint_as_float(byte == 255 ? 0x7FFFFFFFu : byte ? byte << 23 : 0x00400000u);
        T* row = static_cast<T*>(a.values) + (p.row + 32 * u) * a.ldv;
        Pack<T> out;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2_raw h =
                __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(codes[u] >> (8 * k)), __NV_E2M1);
            const float2 f = __half22float2(__half2(h));
            reinterpret_cast<T*>(out.w)[2 * k] = from_f32<T>(f.x * by);
            reinterpret_cast<T*>(out.w)[2 * k + 1] = from_f32<T>(f.y * by);
        }
        if constexpr (!kVec) {
            store_shifted(row, j, a.width, out, here, same_as_next, same_as_last);
        } else if (here && j + 8 <= a.width) {
            store_pack(row + j, out);
        } else if (here) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < a.width)
                    row[j + k] = reinterpret_cast<const T*>(out.w)[k];
        }
    }
}

int check(const mxfp4_args* a)
{
    if (!a)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    if (a->rows < 0 || a->width < 0 || a->rows >= (INT64_C(1) << 31) || a->width >= (INT64_C(1) << 31))
        return fail_with(GEMM_ERR_ARG, "sizes must be in [0, 2^31)");
    if (!type_ok(a->type))
        return fail_with(GEMM_ERR_ARG, "bad type");
    if (a->rows == 0 || a->width == 0)
        return GEMM_OK;
    if (!a->values || !a->codes || !a->scales)
        return fail_with(GEMM_ERR_ARG, "values, codes or scales is NULL");
    if (a->ldv < a->width || a->ldc < (a->width + 31) / 32 * 16)
        return fail_with(GEMM_ERR_ARG, "row stride below the row");
    if (!aligned(a->values, type_bytes(a->type)) || !aligned(a->codes, 16) || a->ldc % 16 != 0 || !aligned(a->scales, 16))
        return fail_with(GEMM_ERR_ALIGN, "values must be aligned to their elements, codes, their rows and scales to 16 bytes");
    return GEMM_OK;
}

template <typename T, bool kQuantize>
cudaError_t launch(const mxfp4_args& a, cudaStream_t s)
{
    Args k{};
    k.rows = a.rows;
    k.width = a.width;
    k.ldv = a.ldv;
    k.ldc = a.ldc;
    k.blocks = static_cast<int>((a.width + 31) / 32);
    k.groups = static_cast<int>((a.width + 127) / 128);
    k.per_row = k.groups >= 16 ? kThreads : k.groups * 16;
    k.chunks = (k.groups * 16 + k.per_row - 1) / k.per_row;
    k.sets = (a.rows + 127) / 128 * 32;
    k.values = a.values;
    k.codes = static_cast<uint8_t*>(a.codes);
    k.scales = static_cast<uint4*>(a.scales);
    const int rows = kThreads / k.per_row;
    const long long grid = (k.sets + rows - 1) / rows * k.chunks;
    if (grid >= (INT64_C(1) << 31))
        return cudaErrorInvalidConfiguration;
    const bool vec = packs(a.values, a.ldv, a.type);
    void (*kernel)(Args);
    if constexpr (kQuantize)
        kernel = vec ? sat_mxfp4_quantize_kernel<T, true> : sat_mxfp4_quantize_kernel<T, false>;
    else
        kernel = vec ? sat_mxfp4_dequantize_kernel<T, true> : sat_mxfp4_dequantize_kernel<T, false>;
    return ffn::launch_early(kernel, static_cast<unsigned>(grid), kThreads, 0, 1, s, k);
}

template <bool kQuantize>
cudaError_t launch_as(const mxfp4_args& a, void* stream)
{
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a.type == GEMM_C_F32    ? launch<float, kQuantize>(a, s)
           : a.type == GEMM_C_BF16 ? launch<__nv_bfloat16, kQuantize>(a, s)
                                   : launch<__half, kQuantize>(a, s);
}

}  // namespace

extern "C" {

int64_t mxfp4_scale_bytes(int64_t rows, int64_t width)
{
    set_last_error("");
    if (rows < 0 || width < 0 || rows >= (INT64_C(1) << 31) || width >= (INT64_C(1) << 31))
        return fail_with(GEMM_ERR_ARG, "sizes must be in [0, 2^31)");
    return (rows + 127) / 128 * ((width + 127) / 128) * 512;
}

int mxfp4_quantize(const mxfp4_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->rows == 0 || args->width == 0)
        return rc;
    const cudaError_t e = launch_as<true>(*args, stream);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the quantisation: %s", cudaGetErrorString(e));
}

int mxfp4_dequantize(const mxfp4_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->rows == 0 || args->width == 0)
        return rc;
    const cudaError_t e = launch_as<false>(*args, stream);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the dequantisation: %s", cudaGetErrorString(e));
}

}  // extern "C"
