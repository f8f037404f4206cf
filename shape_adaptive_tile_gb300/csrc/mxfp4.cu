// Microscaled 4-bit matrices: quantisation and its inverse (include/ffn.h).
#include "ffn.h"

#include <climits>
#include <type_traits>

#include "ffn_device.h"
#include "ffn_ptx.cuh"
#include "ffn_tile.h"
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 256;

struct Args {
    unsigned rows, width, ldv, ldc;  // (rows fit 32 bits together with the 127 that fill up a tile)
    unsigned blocks;   // of 32 columns, of a row
    unsigned groups;   // of four blocks, of a row: one word of scales
    unsigned per_row;  // threads that take a row's columns in one go, eight each: 16 times a number of groups
    unsigned chunks;   // goes that a row takes
    unsigned sets;     // sets of four rows, 32 apart in a tile of 128: their words of scales are 16 consecutive bytes
    unsigned stride;   // sets that all CTAs of a chunk take in one go
    void* values;
    uint8_t* codes;
    uint4* scales;  // by group and row within 32 of a tile
};

// What a thread does in all its sets of rows: columns 8 unit ...
struct Place {
    bool in;
    unsigned unit, first;  // first: the first set
};

__device__ __forceinline__ Place place(const Args& a)
{
    Place p;
    const unsigned go = blockIdx.x / a.chunks, chunk = blockIdx.x - go * a.chunks;
    const unsigned sub = threadIdx.x / a.per_row, rows = kThreads / a.per_row;
    p.unit = chunk * a.per_row + threadIdx.x - sub * a.per_row;
    p.in = sub < rows && p.unit < a.groups * 16;
    p.first = go * rows + sub;
    return p;
}

// The first row of a set, and the place of its scales.
__device__ __forceinline__ unsigned row_of(unsigned set) { return (set >> 5) * 128 + (set & 31); }
__device__ __forceinline__ unsigned long long scales_of(const Args& a, unsigned set, unsigned unit)
{
    return (static_cast<unsigned long long>(set >> 5) * a.groups + (unit >> 4)) * 32 + (set & 31);
}

// Eight elements of row[j ..], one by one; past the width 0.
template <typename T>
__device__ __forceinline__ Pack<T> load_singly(const T* row, long long j, long long width)
{
    Pack<T> v{};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (j + i < width)
            reinterpret_cast<T*>(v.w)[i] = row[j + i];
    return v;
}

// The 16-byte pieces around eight elements of a row that may start off 16 bytes.
// All rows' pieces are on their way before the first is shifted: with each row's
// loads behind a test of its own, 8192 x 8191 bf16 took 58 us instead of 48, and
// 55049 x 427 fp16, with the elements at the rows' ends one by one, 28 instead of
// 22. (fp32 in pairs of rows: 8000 x 4097 44 us; 41 one after the other.)
template <typename T>
struct Around {
    static constexpr int P = 16 / sizeof(T), N = sizeof(T) == 4 ? 3 : 2;
    uint4 q[N];

    // Those that hold an element of the row, whole: what else is in them has to be the matrix's or between its rows. (By
    // coherent loads: the kernel before this one may still write the matrix when this one starts.)
    __device__ __forceinline__ void load(const T* row, long long j, long long width)
    {
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + j)) & 15u;
        const int back = static_cast<int>(off / sizeof(T));
        const uint4* from = reinterpret_cast<const uint4*>(row + j - back);
#pragma unroll
        for (int i = 0; i < N; ++i)
            q[i] = j - back + i * P < width && (i < N - 1 || off) ? from[i] : make_uint4(0, 0, 0, 0);
    }

    // The eight elements, shifted into place; past the width 0.
    __device__ __forceinline__ Pack<T> elements(const T* row, long long j, long long width) const
    {
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + j)) & 15u;
        uint32_t w[4 * N + 3] = {};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[4 * i] = q[i].x;
            w[4 * i + 1] = q[i].y;
            w[4 * i + 2] = q[i].z;
            w[4 * i + 3] = q[i].w;
        }
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            w[i] = off & 4 ? w[i + 1] : w[i];
        Pack<T> v;
#pragma unroll
        for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i)
            v.w[i] = sizeof(T) == 2 && (off & 2) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        if (j + 8 > width) {
            const int left = static_cast<int>(width - j);
#pragma unroll
            for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) {
                if constexpr (sizeof(T) == 4)
                    v.w[i] = i < left ? v.w[i] : 0u;
                else
                    v.w[i] = 2 * i + 1 < left ? v.w[i] : 2 * i < left ? v.w[i] & 0xFFFFu : 0u;
            }
        }
        return v;
    }
};

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
        asm("max.u16x2 %0, %1, %2;" : "=r"(two) : "r"(two), "r"(p.w[k] & 0x7FFF7FFFu));
    const uint16_t top = static_cast<uint16_t>(max(two & 0xFFFFu, two >> 16));
    return __float_as_uint(to_f32(*reinterpret_cast<const T*>(&top))) >> 23;
}

// Eight numbers' codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// Eight columns of four rows a thread at a time, all loads in flight at once:
// four threads a block of 32, sixteen a word of scales. The exponent field of a
// block's largest magnitude is its logarithm rounded down (bits compare as
// magnitudes do); the four rows' fields share a word, whose bytes are compared
// and exchanged together: 4 shuffles for 32 values a thread instead of 16. A CTA
// takes many sets of rows of its columns, so that what a thread works out about
// its place is worked out once. 8192 x 8192 bf16 30.8 us, 81% of the copy rate,
// with some 3 of 4 instructions a cycle; fp32 45 us, 98%.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, !kVec && sizeof(T) == 4 ? 3 : 4) sat_mxfp4_quantize_kernel(const __grid_constant__ Args a)
{
    launch_dependents();
    wait_for_earlier();
    const Place p = place(a);
    const long long j = p.unit * 8ll;
    const int g = threadIdx.x >> 2 & 3;
    const bool coded = (p.unit >> 2) < a.blocks;
    const unsigned sub = threadIdx.x / a.per_row;
#pragma unroll 1
    for (unsigned set = p.first; set - sub < a.sets; set += a.stride) {  // (the same for all of a CTA)
        const bool in = p.in && set < a.sets;
        const unsigned row = row_of(set);
        const T* from = static_cast<const T*>(a.values) + static_cast<unsigned long long>(row) * a.ldv;
        auto row_at = [&](int u) { return from + static_cast<unsigned long long>(32 * u) * a.ldv; };
        Pack<T> v[4];
        if constexpr (kVec) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (in && row + 32 * u < a.rows)
                    v[u] = j + 8 <= a.width ? load_pack(row_at(u) + j) : load_singly(row_at(u), j, a.width);
                else
                    v[u] = Pack<T>{};
        } else {
            // Pieces of the first and the last row may reach out of the matrix, and so may those of rows closer than 16 bytes.
            auto inside = [&](int u) {
                return row + 32 * u > 0 && row + 32 * u + 1 < a.rows && a.ldv >= static_cast<unsigned>(Around<T>::P);
            };
            constexpr int AT_ONCE = sizeof(T) == 4 ? 2 : 4;  // (registers)
#pragma unroll
            for (int u0 = 0; u0 < 4; u0 += AT_ONCE) {
                Around<T> pieces[AT_ONCE];
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u)
                    pieces[u].load(row_at(u0 + u), j, in && inside(u0 + u) ? static_cast<long long>(a.width) : LLONG_MIN);
#pragma unroll
                for (int u = 0; u < AT_ONCE; ++u)
                    if (inside(u0 + u) || !in || row + 32 * (u0 + u) >= a.rows)
                        v[u0 + u] = pieces[u].elements(row_at(u0 + u), j, a.width);
                    else
                        v[u0 + u] = load_singly(row_at(u0 + u), j, a.width);
            }
        }
        uint32_t fields = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            fields |= largest_field(v[u]) << (8 * u);
        fields = __vmaxu4(fields, __shfl_xor_sync(0xffffffffu, fields, 1));
        fields = __vmaxu4(fields, __shfl_xor_sync(0xffffffffu, fields, 2));
        // exponent + 127 of each row's block: two less, not below 0, and 255 for what is not finite.
        const uint32_t bytes = __vsubus4(fields, 0x02020202u) | __vcmpeq4(fields, 0xFFFFFFFFu);
        uint8_t* to = a.codes + static_cast<unsigned long long>(row) * a.ldc + p.unit * 4;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t byte = bytes >> (8 * u) & 255u;
            const float by = __uint_as_float((254u - byte) << 23);  // 2^-exponent, always a normal number (of 255: not used)
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = to_f32(reinterpret_cast<const T*>(v[u].w)[k]) * by;
            const uint32_t w = codes_of(x);
            if (in && coded && row + 32 * u < a.rows)
                *reinterpret_cast<uint32_t*>(to + static_cast<unsigned long long>(32 * u) * a.ldc) = byte == 255 ? 0u : w;
        }
        // The bytes of four blocks x four rows, each block's in one group of lanes, turned: group g gets row g's word.
        uint32_t other = __shfl_xor_sync(0xffffffffu, bytes, 4);
        uint32_t word = __byte_perm(bytes, other, g & 1 ? 0x3715 : 0x6240);
        other = __shfl_xor_sync(0xffffffffu, word, 8);
        word = __byte_perm(word, other, g & 2 ? 0x3276 : 0x5410);
        if (in && (threadIdx.x & 3) == 0)
            reinterpret_cast<uint32_t*>(a.scales + scales_of(a, set, p.unit))[g] = word;  // 0 for rows past the last one
    }
}

// The fp16 numbers of eight codes, the first in the lowest four bits.
__device__ __forceinline__ void numbers_of(uint32_t codes, uint32_t (&two)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(two[0]), "=r"(two[1]), "=r"(two[2]), "=r"(two[3])
        : "r"(codes));
}

// 2^(byte - 127), of byte 0 below the normal numbers; NaN of 255.
__device__ __forceinline__ float power_of(uint32_t byte)
{
    return __uint_as_float(byte == 255 ? 0x7FFFFFFFu : byte ? byte << 23 : 0x00400000u);
}

// Eight elements from their codes, the first `n` by one scale, the others by the next block's.
template <typename T>
__device__ __forceinline__ Pack<T> elements_of(uint32_t codes, float by, float by_next, int n)
{
    uint32_t two[4];
    numbers_of(codes, two);
    Pack<T> out;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two[k]));
        const float x = f.x * (2 * k < n ? by : by_next), y = f.y * (2 * k + 1 < n ? by : by_next);
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float*>(out.w)[2 * k] = x;
            reinterpret_cast<float*>(out.w)[2 * k + 1] = y;
        } else if constexpr (std::is_same_v<T, __half>) {
            reinterpret_cast<__half2*>(out.w)[k] = __floats2half2_rn(x, y);
        } else {
            reinterpret_cast<__nv_bfloat162*>(out.w)[k] = __floats2bfloat162_rn(x, y);
        }
    }
    return out;
}

// Rows that start off 16 bytes: a thread takes the eight elements that begin at
// the first whole 16 bytes among its own, so that it stores whole ones: their
// codes are its own and the next thread's word, shifted (codes are a quarter of
// the elements' bits, and nothing is exchanged), and the last of a block's four
// threads has the next block's scale for the rest. What is before the row's first
// whole 16 bytes, its first thread stores too. 8192 x 8191 bf16 39 us; 61 with
// finished elements exchanged between lanes and shifted, 174 one by one.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) sat_mxfp4_dequantize_kernel(const __grid_constant__ Args a)
{
    launch_dependents();
    wait_for_earlier();
    const Place p = place(a);
    const bool coded = p.in && (p.unit >> 2) < a.blocks, more = ((p.unit + 1) >> 2) < a.blocks;
    const long long j = p.unit * 8ll;
    const unsigned sub = threadIdx.x / a.per_row;
#pragma unroll 1
    for (unsigned set = p.first; set - sub < a.sets; set += a.stride) {
        const bool in = coded && set < a.sets;
        const unsigned row = row_of(set);
        const uint4 s4 = in ? a.scales[scales_of(a, set, p.unit)] : make_uint4(0, 0, 0, 0);
        const uint32_t words[4] = {s4.x, s4.y, s4.z, s4.w};
        uint4 n4 = make_uint4(0, 0, 0, 0);  // of the next four blocks, where the next thread's block is one of them
        if (!kVec && in && more && (p.unit & 15) == 15)
            n4 = a.scales[scales_of(a, set, p.unit + 1)];
        const uint32_t next_words[4] = {n4.x, n4.y, n4.z, n4.w};
        const uint8_t* from = a.codes + static_cast<unsigned long long>(row) * a.ldc + p.unit * 4;
        uint32_t codes[4], next[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool here = in && row + 32 * u < a.rows;
            const uint32_t* at = reinterpret_cast<const uint32_t*>(from + static_cast<unsigned long long>(32 * u) * a.ldc);
            codes[u] = here ? at[0] : 0u;
            next[u] = !kVec && here && more ? at[1] : 0u;
        }
        T* to = static_cast<T*>(a.values) + static_cast<unsigned long long>(row) * a.ldv;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool here = in && row + 32 * u < a.rows;
            if (!kVec && !here)
                break;
            const float by = power_of(words[u] >> (8 * (p.unit / 4 % 4)) & 255u);
            T* at = to + static_cast<unsigned long long>(32 * u) * a.ldv;
            if constexpr (kVec) {
                const Pack<T> out = elements_of<T>(codes[u], by, by, 8);
                if (here && j + 8 <= a.width) {
                    store_pack(at + j, out);
                } else if (here) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (j + k < a.width)
                            at[j + k] = reinterpret_cast<const T*>(out.w)[k];
                }
            } else {
                constexpr int P = 16 / sizeof(T);
                const int skip = -static_cast<int>(reinterpret_cast<uintptr_t>(at) / sizeof(T)) & (P - 1);
                const uint32_t next_byte =
                    ((p.unit & 15) == 15 ? next_words[u] : words[u] >> (8 * ((p.unit + 1) / 4 % 4))) & 255u;
                const Pack<T> out = elements_of<T>(__funnelshift_r(codes[u], next[u], 4 * skip), by, power_of(next_byte),
                                                   (p.unit & 3) == 3 ? 8 - skip : 8);
                const long long first = j + skip;
                if (first + 8 <= a.width) {
#pragma unroll
                    for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k)
                        *reinterpret_cast<uint4*>(at + first + k * P) =
                            make_uint4(out.w[4 * k], out.w[4 * k + 1], out.w[4 * k + 2], out.w[4 * k + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (first + k < a.width)
                            at[first + k] = reinterpret_cast<const T*>(out.w)[k];
                }
                if (p.unit == 0 && skip > 0) {
                    const Pack<T> head = elements_of<T>(codes[u], by, by, 8);
#pragma unroll
                    for (int k = 0; k < P - 1; ++k)
                        if (k < skip && k < a.width)
                            at[k] = reinterpret_cast<const T*>(head.w)[k];
                }
            }
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
    if (a->ldv < a->width || a->ldc < (a->width + 31) / 32 * 16 || a->ldv >= (INT64_C(1) << 31) || a->ldc >= (INT64_C(1) << 31))
        return fail_with(GEMM_ERR_ARG, "row stride below the row, or not below 2^31");
    if (!aligned(a->values, type_bytes(a->type)) || !aligned(a->codes, 16) || a->ldc % 16 != 0 || !aligned(a->scales, 16))
        return fail_with(GEMM_ERR_ALIGN, "values must be aligned to their elements, codes, their rows and scales to 16 bytes");
    return GEMM_OK;
}

template <typename T, bool kQuantize>
cudaError_t launch(const mxfp4_args& a, int sms, cudaStream_t s)
{
    Args k{};
    k.rows = static_cast<unsigned>(a.rows);
    k.width = static_cast<unsigned>(a.width);
    k.ldv = static_cast<unsigned>(a.ldv);
    k.ldc = static_cast<unsigned>(a.ldc);
    k.blocks = (k.width + 31) / 32;
    k.groups = (k.width + 127) / 128;
    k.per_row = k.groups >= 16 ? kThreads : k.groups * 16;
    k.chunks = (k.groups * 16 + k.per_row - 1) / k.per_row;
    k.sets = (k.rows + 127) / 128 * 32;
    k.values = a.values;
    k.codes = static_cast<uint8_t*>(a.codes);
    k.scales = static_cast<uint4*>(a.scales);
    // CTAs with several sets of rows each, or, of many columns, one. Quantising, eight an SM (8192 x 8192 bf16 30.8 us; 32.2
    // with 32), and 32 the other way, whose stores want more of them under way (fp32 45.5 us; 51.0 with eight).
    const unsigned ctas = (kQuantize ? 8u : 32u) * static_cast<unsigned>(sms);
    const unsigned rows = kThreads / k.per_row, goes = (k.sets + rows - 1) / rows;
    const unsigned most = k.chunks >= ctas ? 1 : ctas / k.chunks;
    const unsigned per_chunk = goes < most ? goes : most;
    k.stride = per_chunk * rows;
    const long long grid = static_cast<long long>(per_chunk) * k.chunks;
    const bool vec = packs(a.values, a.ldv, a.type);
    void (*kernel)(Args);
    if constexpr (kQuantize)
        kernel = vec ? sat_mxfp4_quantize_kernel<T, true> : sat_mxfp4_quantize_kernel<T, false>;
    else
        kernel = vec ? sat_mxfp4_dequantize_kernel<T, true> : sat_mxfp4_dequantize_kernel<T, false>;
    return ffn::launch_early(kernel, static_cast<unsigned>(grid), kThreads, 0, 1, s, k);
}

template <bool kQuantize>
int launch_as(const mxfp4_args& a, void* stream, const char* what)
{
    int sms = 0;
    const int rc = ffn::device_sms(&sms);
    if (rc)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a.type == GEMM_C_F32    ? launch<float, kQuantize>(a, sms, s)
                          : a.type == GEMM_C_BF16 ? launch<__nv_bfloat16, kQuantize>(a, sms, s)
                                                  : launch<__half, kQuantize>(a, sms, s);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching the %s: %s", what, cudaGetErrorString(e));
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
    return launch_as<true>(*args, stream, "quantisation");
}

int mxfp4_dequantize(const mxfp4_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->rows == 0 || args->width == 0)
        return rc;
    return launch_as<false>(*args, stream, "dequantisation");
}

}  // extern "C"
