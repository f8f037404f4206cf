// Microscaled 4-bit matrices: quantisation and its inverse (include/ffn.h).
#include <cuda_fp4.h>

#include "ffn.h"
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 256;

struct Args {
    long long rows, width, ldv, ldc;
    long long blocks;  // of 32 columns, of a row
    long long groups;  // of four blocks, of a row: one word of scales
    long long units;   // 8 columns each: rows x 16 groups
    const void* values;
    void* out;
    uint8_t* codes;
    uint32_t* scales;  // a word for each row and group
};

// The word of row r, group g.
__device__ __forceinline__ long long scale_word(long long r, long long g, long long groups)
{
    return (r / 128 * groups + g) * 128 + r % 32 * 4 + r % 128 / 32;
}

// Eight values of row[j ..]; past the width 0.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(float (&v)[8], const T* row, long long j, long long width)
{
    if (kVec && j + 8 <= width) {
        const Pack<T> p = load_pack(row + j);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = to_f32(reinterpret_cast<const T*>(p.w)[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = j + i < width ? to_f32(row[j + i]) : 0.0f;
    }
}

// Eight columns a thread: four threads a block of 32, sixteen a word of
// scales. The block's largest magnitude is compared as bits (past the infinity
// come the NaN), its exponent field is the logarithm rounded down.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) sat_mxfp4_quantize_kernel(const Args a)
{
    const long long unit = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const long long per_row = a.groups * 16, r = unit / per_row, i = unit - r * per_row;
    const bool in = unit < a.units && r < a.rows;
    float v[8];
    if (in)
        load8<T, kVec>(v, static_cast<const T*>(a.values) + r * a.ldv, i * 8, a.width);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        top = max(top, in ? __float_as_uint(v[k]) & 0x7FFFFFFFu : 0u);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t field = top >> 23;
    const bool bad = field == 255;
    const uint32_t byte = bad ? 255u : field > 2 ? field - 2 : 0u;  // exponent + 127
    if (in && i / 4 < a.blocks) {
        const float by = __uint_as_float(bad ? 0u : (254u - byte) << 23);  // 2^-exponent, always a normal number
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 p = bad ? make_float2(0.0f, 0.0f) : make_float2(v[2 * k] * by, v[2 * k + 1] * by);
            w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest)) << (8 * k);
        }
        *reinterpret_cast<uint32_t*>(a.codes + r * a.ldc + i * 4) = w;
    }
    uint32_t word = byte << (8 * (threadIdx.x / 4 % 4));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (unit < a.units && i % 16 == 0)
        a.scales[scale_word(r, i / 16, a.groups)] = word;  // 0 for rows past the last one
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) sat_mxfp4_dequantize_kernel(const Args a)
{
    const long long unit = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const long long per_row = a.blocks * 4, r = unit / per_row, i = unit - r * per_row;
    if (r >= a.rows)
        return;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(a.codes + r * a.ldc + i * 4);
    const uint32_t byte = a.scales[scale_word(r, i / 16, a.groups)] >> (8 * (i / 4 % 4)) & 255u;
    // 2^(byte - 127): of byte 0 it is below the normal numbers.
    const float by = __uint_as_float(byte == 255 ? 0x7FFFFFFFu : byte ? byte << 23 : 0x00400000u);
    T* row = static_cast<T*>(a.out) + r * a.ldv;
    const long long j = i * 8;
    Pack<T> p;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(w >> (8 * k)), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        reinterpret_cast<T*>(p.w)[2 * k] = from_f32<T>(f.x * by);
        reinterpret_cast<T*>(p.w)[2 * k + 1] = from_f32<T>(f.y * by);
    }
    if (kVec && j + 8 <= a.width) {
        store_pack(row + j, p);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k < a.width)
                row[j + k] = reinterpret_cast<const T*>(p.w)[k];
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

Args args_of(const mxfp4_args& a)
{
    Args k{};
    k.rows = a.rows;
    k.width = a.width;
    k.ldv = a.ldv;
    k.ldc = a.ldc;
    k.blocks = (a.width + 31) / 32;
    k.groups = (a.width + 127) / 128;
    k.values = k.out = a.values;
    k.codes = static_cast<uint8_t*>(a.codes);
    k.scales = static_cast<uint32_t*>(a.scales);
    return k;
}

template <typename T>
cudaError_t quantize(const mxfp4_args& a, cudaStream_t s)
{
    Args k = args_of(a);
    k.units = (a.rows + 127) / 128 * 128 * k.groups * 16;
    const long long grid = (k.units + kThreads - 1) / kThreads;
    if (grid >= (INT64_C(1) << 31))
        return cudaErrorInvalidConfiguration;
    if (packs(a.values, a.ldv, a.type))
        sat_mxfp4_quantize_kernel<T, true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(k);
    else
        sat_mxfp4_quantize_kernel<T, false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(k);
    return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize(const mxfp4_args& a, cudaStream_t s)
{
    Args k = args_of(a);
    k.units = a.rows * k.blocks * 4;
    const long long grid = (k.units + kThreads - 1) / kThreads;
    if (grid >= (INT64_C(1) << 31))
        return cudaErrorInvalidConfiguration;
    if (packs(a.values, a.ldv, a.type))
        sat_mxfp4_dequantize_kernel<T, true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(k);
    else
        sat_mxfp4_dequantize_kernel<T, false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(k);
    return cudaGetLastError();
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
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = args->type == GEMM_C_F32    ? quantize<float>(*args, s)
                          : args->type == GEMM_C_BF16 ? quantize<__nv_bfloat16>(*args, s)
                                                      : quantize<__half>(*args, s);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the quantisation: %s", cudaGetErrorString(e));
}

int mxfp4_dequantize(const mxfp4_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->rows == 0 || args->width == 0)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = args->type == GEMM_C_F32    ? dequantize<float>(*args, s)
                          : args->type == GEMM_C_BF16 ? dequantize<__nv_bfloat16>(*args, s)
                                                      : dequantize<__half>(*args, s);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the dequantisation: %s", cudaGetErrorString(e));
}

}  // extern "C"
