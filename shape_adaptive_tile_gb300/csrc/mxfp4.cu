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

template <typename T, bool kVec>
__device__ __forceinline__ Pack<T> load8(const T* row, long long j, long long width)
{
    if (kVec && j + 8 <= width)
        return load_pack(row + j);
    Pack<T> v{};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (j + i < width)
            reinterpret_cast<T*>(v.w)[i] = row[j + i];
    return v;
}

// The bits of the largest magnitude as an fp32 number: of 16-bit types two values at a time.
__device__ __forceinline__ uint32_t magnitude(const Pack<float>& p)
{
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        top = max(top, p.w[k] & 0x7FFFFFFFu);
    return top;
}

template <typename T>
__device__ __forceinline__ uint32_t magnitude(const Pack<T>& p)
{
    uint32_t two = p.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int k = 1; k < 4; ++k)
        two = __vmaxu2(two, p.w[k] & 0x7FFF7FFFu);
    const uint16_t top = static_cast<uint16_t>(max(two & 0xFFFFu, two >> 16));
    return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&top)));
}

// Eight columns of four rows a thread, all loads in flight at once: four
// threads a block of 32, sixteen a word of scales. A block's largest magnitude
// is compared as bits (past the infinity come the NaN); its exponent field is
// the logarithm rounded down.
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
    uint32_t words[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = to_f32(reinterpret_cast<const T*>(in[u].w)[k]);
        uint32_t top = magnitude(in[u]);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t field = top >> 23;
        const bool bad = field == 255;
        const uint32_t byte = bad ? 255u : field > 2 ? field - 2 : 0u;        // exponent + 127
        const float by = __uint_as_float(bad ? 0u : (254u - byte) << 23);     // 2^-exponent, always a normal number
        if (p.in && p.row + 32 * u < a.rows && (p.unit >> 2) < a.blocks) {
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = bad ? make_float2(0.0f, 0.0f) : make_float2(v[2 * k] * by, v[2 * k + 1] * by);
                w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * k);
            }
            *reinterpret_cast<uint32_t*>(a.codes + (p.row + 32 * u) * a.ldc + p.unit * 4) = w;
        }
        uint32_t word = byte << (8 * (threadIdx.x / 4 % 4));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        words[u] = word;  // 0 for rows past the last one
    }
    if (p.in && threadIdx.x % 16 == 0)
        a.scales[p.at] = make_uint4(words[0], words[1], words[2], words[3]);
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) sat_mxfp4_dequantize_kernel(const __grid_constant__ Args a)
{
    launch_dependents();
    wait_for_earlier();
    const Place p = place(a);
    if (!p.in || (p.unit >> 2) >= a.blocks)
        return;
    const long long j = p.unit * 8ll;
    const uint4 s4 = a.scales[p.at];
    const uint32_t words[4] = {s4.x, s4.y, s4.z, s4.w};
    uint32_t codes[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        codes[u] = p.row + 32 * u < a.rows
                       ? *reinterpret_cast<const uint32_t*>(a.codes + (p.row + 32 * u) * a.ldc + p.unit * 4)
                       : 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        if (p.row + 32 * u >= a.rows)
            return;
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
        if (kVec && j + 8 <= a.width) {
            store_pack(row + j, out);
        } else {
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
