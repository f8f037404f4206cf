// The gated product, its gradients and the products of microscaled matrices
// (include/ffn.h): checks of arguments, tensor maps, and the choice of a tile
// kernel (ffn_tile.cuh).
#include "ffn.h"

#include <algorithm>
#include <mutex>

#include "ffn_device.h"
#include "ffn_tile.cuh"
#include "rows.cuh"

namespace sat {
namespace ffn {

extern const Variant kHalfTiles[], kGradTiles[], kScaledTiles[];
extern const int kNumHalfTiles, kNumGradTiles, kNumScaledTiles;

const Variant* find_variant(int mx, int epi, int cg, int bn, int p_mn, int q_mn, int swap)
{
    const Variant* tab[3] = {kHalfTiles, kGradTiles, kScaledTiles};
    const int num[3] = {kNumHalfTiles, kNumGradTiles, kNumScaledTiles};
    for (int g = 0; g < 3; ++g)
        for (int i = 0; i < num[g]; ++i) {
            const Variant& v = tab[g][i];
            if (v.mx == mx && v.epi == epi && v.cg == cg && v.bn == bn && v.p_mn == p_mn && v.q_mn == q_mn && v.swap == swap)
                return &v;
        }
    return nullptr;
}

}  // namespace ffn
}  // namespace sat

namespace {

using namespace sat;
using namespace sat::rows;
using namespace sat::ffn;

constexpr int64_t kMost = INT64_C(1) << 31;

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t ceil_div(int64_t n, int64_t by) { return (n + by - 1) / by; }

// One factor of a product: `extent` rows (or columns) of the output by k. mn:
// extent is the contiguous one, else k is. Two pointers: two segments of k, two
// products of a batch, or the gate's and the other weights.
struct Factor {
    const void* at[2];
    int64_t ld, extent;
    bool mn;
    const void* scales[2];
    int64_t ld1 = 0;  // the second one's stride, where it is another
};

struct Product {
    int epi, mx;
    Factor x, w;        // x gives the output's rows, w its columns
    bool w_is_weights;  // w may be the first operand for a few rows
    int64_t k;          // of one segment
    int segments, batch;
    int type;           // of 16-bit operands
    int activation, keep, add, out_type;
    float alpha;
    int64_t rows, cols;  // of one output
    void* out[3];
    int64_t ld[3];
    bool beside;  // needs nothing of the kernel before it
    bool padded;  // the outputs' rows go on to a whole number of 16 bytes that nobody reads
    const void* dh;
    int64_t lddh;
};

int map_error(int rc)
{
    return rc == -1 ? fail_with(GEMM_ERR_LAUNCH, "cuTensorMapEncodeTiled is not available from the driver")
                    : fail_with(GEMM_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", rc);
}

CUtensorMapDataType map_type(int type)
{
    return type == GEMM_C_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
           : type == GEMM_C_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

int encode_factor(CUtensorMap* map, const Product& p, const Factor& f, int i, int box_rows)
{
    const uint64_t extent = static_cast<uint64_t>(f.extent), k = static_cast<uint64_t>(p.k), ld = static_cast<uint64_t>(i && f.ld1 ? f.ld1 : f.ld);
    int rc;
    if (p.mx)
        rc = encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, f.at[i], (k + 31) / 32 * 16, extent, ld, 128,
                        static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
    else if (f.mn)
        rc = encode_map(map, map_type(p.type), 2, f.at[i], extent, k, ld, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    else
        rc = encode_map(map, map_type(p.type), 2, f.at[i], k, extent, ld, 64, static_cast<uint32_t>(box_rows),
                        CU_TENSOR_MAP_SWIZZLE_128B);
    return rc ? map_error(rc) : GEMM_OK;
}

// Scales as rows of 512 bytes, one for each tile of 128 rows x 4 blocks, read two at a time.
int encode_scales(CUtensorMap* map, const Product& p, const Factor& f, int i)
{
    const int rc = encode_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, f.scales[i], 128,
                              static_cast<uint64_t>(ceil_div(f.extent, 128) * ceil_div(p.k, 128)), 128, 128, 2,
                              CU_TENSOR_MAP_SWIZZLE_NONE);
    return rc ? map_error(rc) : GEMM_OK;
}

// A launch: its variant, tiles, and the CTAs that share a tile's k (or make a pair).
struct Choice {
    const Variant* v;
    int64_t tp, tq;
    int cluster;
    double us;
    cudaError_t error;
};

// How long a kind of tile takes, in us: a launch with its first loads and last
// stores, a tile's own overhead, a k-block, and adding up the sums of a tile that
// CTAs share, once and for each of them. Measured on a GB300 over 65 to 2048 rows
// and 64 to 16384 of k, of which these give the times to 10% or so, 20% at worst.
// What they decide: of 256 x 1024 by 8192 of k, 17 us as 16 tiles of 128 x 128
// shared by 4 CTAs against 36 unshared and 41 as 4 pairs' tiles; of 2048 x 2048 by
// 4096, 24 us as 64 pairs' tiles against 37; gated, 1024 x 1024 of 1024 outputs, 8.6
// us as 128 single tiles against 10.0.
struct Cost {
    double launch, tile, block, join, share;
};

Cost cost_of(int mx, bool gated, int cg)
{
    if (cg == 2)
        return mx ? Cost{5.0, 2.2, 0.28, 0.0, 0.0} : Cost{4.5, 1.1, 0.27, 0.0, 0.0};
    if (mx)
        return gated ? Cost{1.0, 6.0, 0.455, 2.4, 0.35} : Cost{1.4, 3.8, 0.32, 1.2, 0.45};
    return Cost{2.0, 2.5, 0.225, 0.8, 0.65};
}

Choice tiles_of(const Product& p, const Variant* v, int sms)
{
    const bool gated = p.epi != kStore;
    Choice c{v, 0, 0, v->cg, 0.0, cudaSuccess};
    if (v->swap) {
        c.tp = ceil_div(p.cols, 128);
        c.tq = ceil_div(p.rows, v->bn);
    } else {
        c.tp = ceil_div(p.rows, 128 * v->cg);
        c.tq = ceil_div(p.cols, gated ? v->bn / 2 : v->bn);
    }
    const int64_t tiles = c.tp * c.tq * p.batch, num_kb = ceil_div(p.k, p.mx ? 256 : 64) * p.segments;
    if (v->swap) {
        // Every SM wants a CTA: all of them together keep the memory busy. Of 4-bit weights two, as their rings are short
        // (8192 x 8192 gated by one token: 16.4 us as 256 CTAs, 23.1 as 128; 16-bit weights lose 1 to 3%). At least four
        // k-blocks a CTA, and the sums have to fit in the ring.
        const int64_t ctas = p.mx && v->bn <= 32 ? 2 * sms : sms;
        // Two CTAs an SM for up to 32 tokens, where the runtime counts one all the same: twice what it says of the tiles of 64
        // tokens, which fill an SM (8192 x 8192 by one token: 9.6 us in clusters of four, 10.2 in clusters of two).
        const int per_sm = v->bn <= 32 ? 2 : 1;
        const Variant* full = per_sm == 1 ? v : find_variant(v->mx, v->epi, 1, 64, v->p_mn, v->q_mn, 1);
        int64_t s = 1;
        for (int64_t n = 2; n <= 8 && tiles * n <= ctas && num_kb / n >= 4; ++n) {
            if ((n - 1) * ceil_div(v->chunks, n) * v->part_bytes > v->ring_bytes)
                continue;
            int fit = 0;
            if ((c.error = full->fit(static_cast<int>(n), &fit)) != cudaSuccess)
                return c;
            if (tiles <= per_sm * fit)
                s = n;
        }
        c.cluster = static_cast<int>(s);
        return c;
    }
    const Cost t = cost_of(p.mx, gated, v->cg);
    if (v->persistent) {
        c.us = t.launch + ceil_div(tiles, sms / v->cg) * (t.tile + t.block * num_kb);
        return c;
    }
    for (int64_t s = 1; s <= 8 && s <= std::max<int64_t>(1, num_kb / 4); ++s) {
        if ((s - 1) * ceil_div(v->chunks, s) * v->part_bytes > v->ring_bytes)
            continue;
        int fit = sms;
        if (s > 1 && (c.error = v->fit(static_cast<int>(s), &fit)) != cudaSuccess)
            return c;
        if (fit < 1)
            continue;
        const double us = t.launch + ceil_div(tiles, fit) * (t.tile + t.block * ceil_div(num_kb, s) + (s > 1 ? t.join + t.share * s : 0.0));
        if (s == 1 || us < c.us) {
            c.cluster = static_cast<int>(s);
            c.us = us;
        }
    }
    return c;
}

int launch_product(const Product& p, int sms, cudaStream_t stream)
{
    const bool gated = p.epi != kStore;
    const int64_t num_kb = ceil_div(p.k, p.mx ? 256 : 64) * p.segments;
    // A few rows: the weights are the first operand, so that no accumulator row goes unused.
    const bool swap = p.w_is_weights && p.rows <= 64;
    Choice c;
    if (swap) {
        c = tiles_of(p, find_variant(p.mx, p.epi, 1, p.rows <= 16 ? 16 : p.rows <= 32 ? 32 : 64, p.w.mn, p.x.mn, 1), sms);
    } else {
        c = tiles_of(p, find_variant(p.mx, p.epi, 2, 256, p.x.mn, p.w.mn, 0), sms);
        const Choice one = tiles_of(p, find_variant(p.mx, p.epi, 1, p.mx && gated ? 256 : 128, p.x.mn, p.w.mn, 0), sms);
        if (one.error != cudaSuccess || one.us < c.us)
            c = one;
    }
    if (c.error != cudaSuccess)
        return fail_with(GEMM_ERR_LAUNCH, "asking for a tile kernel's clusters: %s", cudaGetErrorString(c.error));
    const Variant* v = c.v;
    const int cluster = c.cluster;
    const int64_t tp = c.tp, tq = c.tq, tiles = tp * tq * p.batch;
    // (The kernels count tiles, and a CTA's k-blocks, in 32 bits; at a quarter of a microsecond each that is minutes.)
    if (tiles * 16 >= kMost || ceil_div(tiles, sms / 2) * num_kb >= kMost)
        return fail_with(GEMM_ERR_ARG, "too many tiles");
    const int grid = static_cast<int>(v->persistent ? std::min<int64_t>(tiles, sms / v->cg) * v->cg : tiles * cluster);
    TileArgs a{};
    a.tiles_p = static_cast<int>(tp);
    a.tiles_q = static_cast<int>(tq);
    a.batch = p.batch;
    a.num_kb = static_cast<int>(num_kb);
    a.seg_kb = static_cast<int>(num_kb / p.segments);
    a.tail_steps = p.mx ? static_cast<int>(ceil_div(p.k - (num_kb - 1) * 256, 64)) : 4;
    a.kb_per_rank = v->persistent ? a.num_kb : static_cast<int>(std::max<int64_t>(1, ceil_div(num_kb, cluster)));
    a.group = v->cg == 2 ? 8 : 16;
    a.idesc = p.mx ? idesc_mxf4(128 * v->cg, v->bn)
                   : idesc_f32acc(p.type == GEMM_C_BF16 ? kFmtBF16 : kFmtF16, 128 * v->cg, v->bn, v->q_mn != 0, v->p_mn != 0);
    a.alpha = p.alpha;
    a.activation = p.activation;
    a.out_kind = p.out_type;
    a.add = p.add;
    a.keep = p.keep;
    a.beside = p.beside;
    a.rows = static_cast<int>(p.rows);
    a.cols = static_cast<int>(p.cols);
    const int outs = p.epi == kStore ? p.batch : p.epi == kGrad ? 2 : p.keep ? 3 : 1;
    TileMaps m{};
    ScaleMaps sm{};
    const Factor &first = swap ? p.w : p.x, &second = swap ? p.x : p.w;
    const int qbox = std::min(64, v->bn / v->cg);
    // The second pointers: of a gated product the weights' only; of segments or a batch both factors'.
    const bool two_first = gated ? swap : p.segments * p.batch > 1, two_second = gated ? !swap : p.segments * p.batch > 1;
    int rc = GEMM_OK;
    for (int i = 0; i < 2 && !rc; ++i) {
        if (i == 0 || two_first)
            rc = encode_factor(&m.p[i], p, first, i, 128);
        if (!rc && (i == 0 || two_second))
            rc = encode_factor(&m.q[i], p, second, i, qbox);
        if (p.mx) {
            if (!rc && (i == 0 || two_first))
                rc = encode_scales(&sm.p[i], p, first, i);
            if (!rc && (i == 0 || two_second))
                rc = encode_scales(&sm.q[i], p, second, i);
        }
    }
    a.sf_rows_p = a.sf_rows_q = p.mx ? static_cast<int>(ceil_div(p.k, 128)) : 0;
    const int es = type_bytes(p.out_type);
    for (int i = 0; i < outs && !rc; ++i) {
        a.out[i] = p.out[i];
        a.ld[i] = p.ld[i];
        if (!swap && aligned(p.out[i], 16) && p.ld[i] * es % 16 == 0) {
            a.tma_out |= 1 << i;
            if (p.padded || p.cols * es % 16 == 0)
                a.tma_edge |= 1 << i;
            const int e = encode_map(&m.o[i], map_type(p.out_type), es, p.out[i], static_cast<uint64_t>(p.cols),
                                     static_cast<uint64_t>(p.rows), static_cast<uint64_t>(p.ld[i]), static_cast<uint32_t>(128 / es),
                                     32, CU_TENSOR_MAP_SWIZZLE_128B);
            rc = e ? map_error(e) : GEMM_OK;
        }
    }
    if (!rc && p.epi == kGrad) {
        const int e = encode_map(&m.o[2], map_type(p.type), 2, p.dh, static_cast<uint64_t>(p.cols), static_cast<uint64_t>(p.rows),
                                 static_cast<uint64_t>(p.lddh), 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
        rc = e ? map_error(e) : GEMM_OK;
    }
    if (rc)
        return rc;
    const cudaError_t e = v->launch(m, p.mx ? &sm : nullptr, a, grid, cluster, stream);
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "launching a tile kernel: %s", cudaGetErrorString(e));
}

// ---- gated product ------------------------------------------------------------

bool rows16(const void* p, int64_t ld) { return aligned(p, 16) && ld * 2 % 16 == 0; }

// A copy's row stride in elements: whole 128-byte lines, an odd number of them (rows do not repeat at a power of two).
int64_t packed_ld(int64_t n)
{
    const int64_t lines = ceil_div(n * 2, 128);
    return (lines | 1) * 64;
}

// What is copied into aligned rows first, and where: byte offsets into the workspace.
struct Copies {
    bool x, w, dh;
    int64_t ldx, ldw, lddh;
    int64_t at_x, at_w, at_w2, at_dh, end;
};

Copies copies_of(const ffn_gated_args& a, const void* dh, int64_t lddh, bool uses_x, bool uses_w, int64_t at)
{
    Copies k{};
    k.x = uses_x && !rows16(a.x, a.ldx);
    k.w = uses_w && (!rows16(a.w, a.ldw) || (!a.w_by_output && a.hidden % 8 != 0));
    k.dh = dh && !rows16(dh, lddh);
    if (k.x) {
        k.ldx = packed_ld(a.width);
        k.at_x = at;
        at += a.rows * k.ldx * 2;
    }
    if (k.w) {
        k.ldw = packed_ld(a.w_by_output ? a.width : a.hidden);
        k.at_w = at;
        k.at_w2 = at + (a.w_by_output ? a.hidden : a.width) * k.ldw * 2;
        at += 2 * (a.w_by_output ? a.hidden : a.width) * k.ldw * 2;
    }
    if (k.dh) {
        k.lddh = packed_ld(a.hidden);
        k.at_dh = at;
        at += a.rows * k.lddh * 2;
    }
    k.end = at;
    return k;
}

int check(const ffn_gated_args* a)
{
    if (!a)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    if (a->rows < 0 || a->width < 0 || a->hidden < 0 || a->rows >= kMost || a->width >= kMost || a->hidden >= kMost / 2)
        return fail_with(GEMM_ERR_ARG, "sizes must be in [0, 2^31), and so must 2 hidden");
    // (Bytes and offsets are counted in 64 bits.)
    if (std::max({a->rows * a->width, a->rows * a->hidden, a->width * a->hidden}) >= INT64_C(1) << 56)
        return fail_with(GEMM_ERR_ARG, "a matrix of 2^56 elements or more");
    if (a->type != GEMM_C_BF16 && a->type != GEMM_C_F16)
        return fail_with(GEMM_ERR_ARG, "type must be bf16 or fp16");
    if (a->activation < FFN_NONE || a->activation > FFN_RELU)
        return fail_with(GEMM_ERR_ARG, "unknown activation %d", a->activation);
    if (a->rows > 0 && a->width > 0 && a->hidden > 0) {
        if (!a->x || !a->w)
            return fail_with(GEMM_ERR_ARG, "x or w is NULL");
        if (a->ldx < a->width || a->ldw < (a->w_by_output ? a->width : 2 * a->hidden))
            return fail_with(GEMM_ERR_ARG, "row stride of x or w below the row");
        if (!aligned(a->x, 2) || !aligned(a->w, 2))
            return fail_with(GEMM_ERR_ALIGN, "x or w is not aligned to its elements");
    }
    if (a->rows > 0 && a->hidden > 0 && a->preact) {
        if (a->ldp < 2 * a->hidden)
            return fail_with(GEMM_ERR_ARG, "row stride of preact below the row");
        if (!aligned(a->preact, 2))
            return fail_with(GEMM_ERR_ALIGN, "preact is not aligned to its elements");
    }
    if (a->ldx >= kMost || a->ldw >= kMost || a->ldp >= kMost || a->ldh >= kMost)
        return fail_with(GEMM_ERR_ARG, "row strides must be below 2^31");
    return GEMM_OK;
}

int check_workspace(const void* at, int64_t bytes, int64_t need, const char* fn)
{
    if (need == 0)
        return GEMM_OK;
    if (!at || bytes < need)
        return fail_with(GEMM_ERR_ARG, "workspace is NULL or below %s()", fn);
    if (!aligned(at, 16))
        return fail_with(GEMM_ERR_ALIGN, "workspace is not aligned to 16 bytes");
    return GEMM_OK;
}

int cuda_rc(cudaError_t e, const char* what)
{
    return e == cudaSuccess ? GEMM_OK : fail_with(GEMM_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
}

// Up to four matrices copied into rows that start on 16 bytes: 16 bytes a
// thread, from the words that hold them. Columns past a row's end are 0. One
// launch for all of them, as of matrices of a few megabytes the launch is most of
// it: 4 us of 14 MB (2047 x 1000 and 1000 x 5002) between other kernels, 9 alone.
struct Copy {
    const uint8_t* from;
    uint8_t* to;
    long long ld, ld_to, bytes;  // of rows: bytes apart, in them
    long long pieces, end;       // 16-byte pieces of a row, and of this matrix and those before it
};
struct CopyArgs {
    Copy m[4];
    int n;
};

__global__ void __launch_bounds__(256) sat_ffn_copy_kernel(const __grid_constant__ CopyArgs a)
{
    wait_for_earlier();
    launch_dependents();
    long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    int k = 0;
    while (k < a.n && i >= a.m[k].end)
        ++k;
    if (k == a.n)
        return;
    const Copy& m = a.m[k];
    if (k > 0)
        i -= a.m[k - 1].end;
    const long long r = i / m.pieces, at = (i - r * m.pieces) * 16;
    const uint8_t* from = m.from + r * m.ld + at;
    const long long left = m.bytes - at;  // > 0
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 2);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(from - odd);
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j)  // (a word that holds a byte of the row is read whole)
        w[j] = 4 * j - odd < left && (j < 4 || odd) ? words[j] : 0u;
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        out[j] = odd ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
        if (left < 4 * j + 4)
            out[j] = left > 4 * j ? out[j] & 0xFFFFu : 0u;
    }
    *reinterpret_cast<uint4*>(m.to + r * m.ld_to + at) = make_uint4(out[0], out[1], out[2], out[3]);
}

// Copies what needs it, and gives x, the weights and dh as they are read.
int pack(const ffn_gated_args& a, const Copies& k, const void* dh, int64_t lddh, void* workspace, cudaStream_t s, Factor* x,
         Factor* w, Factor* d)
{
    char* ws = static_cast<char*>(workspace);
    CopyArgs c{};
    auto add = [&](const void* from, int64_t ld, int64_t to, int64_t ld_to, int64_t rows, int64_t width) {
        Copy& m = c.m[c.n];
        m.from = static_cast<const uint8_t*>(from);
        m.to = reinterpret_cast<uint8_t*>(ws + to);
        m.ld = ld * 2;
        m.ld_to = ld_to * 2;
        m.bytes = width * 2;
        m.pieces = ceil_div(m.bytes, 16);
        m.end = (c.n ? c.m[c.n - 1].end : 0) + rows * m.pieces;
        ++c.n;
        return static_cast<const void*>(m.to);
    };
    x->at[0] = a.x;
    x->ld = a.ldx;
    if (k.x) {
        x->at[0] = add(a.x, a.ldx, k.at_x, k.ldx, a.rows, a.width);
        x->ld = k.ldx;
    }
    const int64_t half = a.w_by_output ? a.hidden * a.ldw * 2 : a.hidden * 2;  // bytes from the gate's weights to the others
    w->at[0] = a.w;
    w->at[1] = static_cast<const char*>(a.w) + half;
    w->ld = a.ldw;
    if (k.w) {
        for (int i = 0; i < 2; ++i)
            w->at[i] = add(w->at[i], a.ldw, i ? k.at_w2 : k.at_w, k.ldw, a.w_by_output ? a.hidden : a.width,
                           a.w_by_output ? a.width : a.hidden);
        w->ld = k.ldw;
    }
    d->at[0] = dh;
    d->ld = lddh;
    if (k.dh) {
        d->at[0] = add(dh, lddh, k.at_dh, k.lddh, a.rows, a.hidden);
        d->ld = k.lddh;
    }
    if (c.n == 0)
        return GEMM_OK;
    const int64_t grid = ceil_div(c.m[c.n - 1].end, 256);
    if (grid >= kMost)
        return fail_with(GEMM_ERR_ARG, "too much to copy into aligned rows");
    return cuda_rc(launch_early(sat_ffn_copy_kernel, static_cast<unsigned>(grid), 256, 0, 1, s, c),
                   "launching a copy into aligned rows");
}

// dg and du of eight columns a thread, from the pre-activations. Memory bounds it: 4096 x 8192 in 59 us, 5.7 TB/s.
struct SlopeArgs {
    long long rows, hidden, units;  // units: eight columns
    const void* dh;
    const void* preact;
    void* dz;  // [dg du], the second half `half` elements after the first
    long long lddh, ldp, ldz, half;
    int activation, beside;
};

// Eight elements, or the `left` that there are; off 16 bytes from the words that hold them.
template <typename T>
__device__ __forceinline__ Pack<T> load_at(const T* p, long long left, bool vec)
{
    if (vec && left >= 8)
        return load_pack(p);
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) >> 1 & 1);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(p - odd);
    uint32_t w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j)
        w[j] = 2 * j - odd < left && (j < 4 || odd) ? words[j] : 0u;
    Pack<T> v;
#pragma unroll
    for (int j = 0; j < 4; ++j)  // (what is past the last element is not looked at)
        v.w[j] = odd ? __funnelshift_r(w[j], w[j + 1], 16) : w[j];
    return v;
}

template <typename T>
__global__ void __launch_bounds__(256) sat_ffn_slope_kernel(const SlopeArgs a, const bool dh_vec, const bool p_vec)
{
    launch_dependents();  // (the next one waits)
    if (!a.beside)
        wait_for_earlier();
    const long long unit = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long r = unit / a.units, j = (unit - r * a.units) * 8;
    if (r >= a.rows) {
        wait_for_earlier();
        return;
    }
    const long long left = a.hidden - j;
    const T* pre = static_cast<const T*>(a.preact) + r * a.ldp + j;
    const Pack<T> d = load_at(static_cast<const T*>(a.dh) + r * a.lddh + j, left, dh_vec);
    const Pack<T> g = load_at(pre, left, p_vec), u = load_at(pre + a.hidden, left, p_vec);
    Pack<T> dg, du;
    with_act(a.activation, [&](auto k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float dv = to_f32(reinterpret_cast<const T*>(d.w)[i]);
            float v, slope;
            act_grad<decltype(k)::value, false>(to_f32(reinterpret_cast<const T*>(g.w)[i]), v, slope);
            reinterpret_cast<T*>(dg.w)[i] = from_f32<T>(dv * to_f32(reinterpret_cast<const T*>(u.w)[i]) * slope);
            reinterpret_cast<T*>(du.w)[i] = from_f32<T>(dv * v);
        }
    });
    // Rows of dz are whole eights of columns: what lies past `hidden` is never read.
    T* z = static_cast<T*>(a.dz) + r * a.ldz + j;
    store_pack(z, dg);
    store_pack(z + a.half, du);
    wait_for_earlier();
}

template <typename T>
cudaError_t launch_slope(const SlopeArgs& a, cudaStream_t s)
{
    const bool dh_vec = aligned(a.dh, 16) && a.lddh % 8 == 0;
    const bool p_vec = aligned(a.preact, 16) && a.ldp % 8 == 0 && a.hidden % 8 == 0;
    const long long grid = ceil_div(a.rows * a.units, 256);
    if (grid >= kMost)
        return cudaErrorInvalidConfiguration;
    return launch_early(sat_ffn_slope_kernel<T>, static_cast<unsigned>(grid), 256, 0, 1, s, a, dh_vec, p_vec);
}

int check_backward(const ffn_gated_args* a, const ffn_gated_grads* g)
{
    const int rc = check(a);
    if (rc)
        return rc;
    if (!g)
        return fail_with(GEMM_ERR_ARG, "grads is NULL");
    if (g->dw_type != GEMM_C_F32 && g->dw_type != a->type && g->dw)
        return fail_with(GEMM_ERR_ARG, "dw_type must be fp32 or args->type");
    if (g->accumulate && g->dw && g->dw_type != GEMM_C_F32)
        return fail_with(GEMM_ERR_ARG, "accumulate needs dw in fp32");
    if (a->rows > 0 && a->hidden > 0 && (g->dx || g->dw) && a->width > 0) {
        if (!g->dh)
            return fail_with(GEMM_ERR_ARG, "dh is NULL");
        if (g->lddh < a->hidden)
            return fail_with(GEMM_ERR_ARG, "row stride of dh below the row");
        if (!aligned(g->dh, 2))
            return fail_with(GEMM_ERR_ALIGN, "dh is not aligned to its elements");
    }
    if (g->dx && a->rows > 0 && a->width > 0 && g->lddx < a->width)
        return fail_with(GEMM_ERR_ARG, "row stride of dx below the row");
    if (g->dw && a->width > 0 && a->hidden > 0 && g->lddw < (a->w_by_output ? a->width : 2 * a->hidden))
        return fail_with(GEMM_ERR_ARG, "row stride of dw below the row");
    if (!aligned(g->dx, 2) || (g->dw && !aligned(g->dw, type_bytes(g->dw_type))))
        return fail_with(GEMM_ERR_ALIGN, "dx or dw is not aligned to its elements");
    if (g->lddh >= kMost || g->lddx >= kMost || g->lddw >= kMost)
        return fail_with(GEMM_ERR_ARG, "row strides must be below 2^31");
    return GEMM_OK;
}

// The backward pass's workspace: [dg du] with both halves' rows on 16 bytes, then copies.
int64_t dz_ld(const ffn_gated_args& a) { return 2 * round_up(a.hidden, 8); }

Copies backward_copies(const ffn_gated_args& a, const ffn_gated_grads& g)
{
    return copies_of(a, a.preact ? nullptr : g.dh, g.lddh, !a.preact || g.dw, !a.preact || g.dx,
                     round_up(a.rows * dz_ld(a) * 2, 128));
}

bool backward_empty(const ffn_gated_args& a, const ffn_gated_grads& g)
{
    return a.rows == 0 || a.width == 0 || a.hidden == 0 || (!g.dx && !g.dw);
}

}  // namespace

extern "C" {

int64_t ffn_gated_workspace(const ffn_gated_args* args)
{
    set_last_error("");
    const int rc = check(args);
    if (rc)
        return rc;
    if (args->rows == 0 || args->width == 0 || args->hidden == 0)
        return 0;
    return copies_of(*args, nullptr, 0, true, true, 0).end;
}

int ffn_gated(const ffn_gated_args* args, void* stream)
{
    set_last_error("");
    int rc = check(args);
    if (rc || args->rows == 0 || args->hidden == 0)
        return rc;
    const ffn_gated_args& a = *args;
    if (!a.h)
        return fail_with(GEMM_ERR_ARG, "h is NULL");
    if (a.ldh < a.hidden)
        return fail_with(GEMM_ERR_ARG, "row stride of h below the row");
    if (!aligned(a.h, 2))
        return fail_with(GEMM_ERR_ALIGN, "h is not aligned to its elements");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.width == 0) {  // a(0) 0 = 0 for every activation
        cudaError_t e = cudaMemset2DAsync(a.h, a.ldh * 2, 0, a.hidden * 2, a.rows, s);
        if (e == cudaSuccess && a.preact)
            e = cudaMemset2DAsync(a.preact, a.ldp * 2, 0, a.hidden * 4, a.rows, s);
        return cuda_rc(e, "clearing h");
    }
    const Copies k = copies_of(a, nullptr, 0, true, true, 0);
    rc = check_workspace(a.workspace, a.workspace_bytes, k.end, "ffn_gated_workspace");
    int sms = 0;
    if (!rc)
        rc = device_sms(&sms);
    if (rc)
        return rc;
    Product p{};
    Factor none{};
    p.epi = kGated;
    rc = pack(a, k, nullptr, 0, a.workspace, s, &p.x, &p.w, &none);
    if (rc)
        return rc;
    p.x.extent = a.rows;
    p.w.extent = a.hidden;
    p.w.mn = !a.w_by_output;
    p.w_is_weights = true;
    p.k = a.width;
    p.segments = p.batch = 1;
    p.type = p.out_type = a.type;
    p.activation = a.activation;
    p.keep = a.preact != nullptr;
    p.alpha = 1.0f;
    p.rows = a.rows;
    p.cols = a.hidden;
    p.out[0] = a.h;
    p.ld[0] = a.ldh;
    p.out[1] = a.preact;
    p.out[2] = a.preact ? static_cast<uint16_t*>(a.preact) + a.hidden : nullptr;
    p.ld[1] = p.ld[2] = a.ldp;
    return launch_product(p, sms, s);
}

int64_t ffn_gated_backward_workspace(const ffn_gated_args* args, const ffn_gated_grads* grads)
{
    set_last_error("");
    const int rc = check_backward(args, grads);
    if (rc)
        return rc;
    return backward_empty(*args, *grads) ? 0 : backward_copies(*args, *grads).end;
}

int ffn_gated_backward(const ffn_gated_args* args, const ffn_gated_grads* grads, void* stream)
{
    set_last_error("");
    int rc = check_backward(args, grads);
    if (rc)
        return rc;
    const ffn_gated_args& a = *args;
    const ffn_gated_grads& g = *grads;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (backward_empty(a, g)) {
        cudaError_t e = cudaSuccess;
        if (g.dx && a.rows > 0 && a.width > 0)  // hidden == 0
            e = cudaMemset2DAsync(g.dx, g.lddx * 2, 0, a.width * 2, a.rows, s);
        if (e == cudaSuccess && g.dw && !g.accumulate && a.width > 0 && a.hidden > 0) {  // rows == 0
            const int64_t es = type_bytes(g.dw_type), cols = a.w_by_output ? a.width : 2 * a.hidden;
            e = cudaMemset2DAsync(g.dw, g.lddw * es, 0, cols * es, a.w_by_output ? 2 * a.hidden : a.width, s);
        }
        return cuda_rc(e, "clearing the gradients");
    }
    const Copies k = backward_copies(a, g);
    rc = check_workspace(g.workspace, g.workspace_bytes, k.end, "ffn_gated_backward_workspace");
    int sms = 0;
    if (!rc)
        rc = device_sms(&sms);
    if (rc)
        return rc;
    Factor x{}, w{}, dh{};
    rc = pack(a, k, a.preact ? nullptr : g.dh, g.lddh, g.workspace, s, &x, &w, &dh);
    if (rc)
        return rc;
    const int64_t ldz = dz_ld(a), half = ldz / 2;
    uint16_t* dz = static_cast<uint16_t*>(g.workspace);
    x.extent = a.rows;
    w.extent = a.hidden;
    w.mn = !a.w_by_output;
    Product p{};
    p.type = p.out_type = a.type;
    p.activation = a.activation;
    p.alpha = 1.0f;
    p.segments = p.batch = 1;
    if (a.preact) {
        SlopeArgs sl{};
        sl.rows = a.rows;
        sl.hidden = a.hidden;
        sl.units = half / 8;
        sl.dh = g.dh;
        sl.lddh = g.lddh;
        sl.preact = a.preact;
        sl.ldp = a.ldp;
        sl.dz = dz;
        sl.ldz = ldz;
        sl.half = half;
        sl.activation = a.activation;
        sl.beside = k.x || k.w;  // the copies are of x and w
        rc = cuda_rc(a.type == GEMM_C_BF16 ? launch_slope<__nv_bfloat16>(sl, s) : launch_slope<__half>(sl, s),
                     "launching the activation's gradient");
    } else {
        p.epi = kGrad;
        p.x = x;
        p.w = w;
        p.k = a.width;
        p.rows = a.rows;
        p.cols = a.hidden;
        p.out[0] = dz;
        p.out[1] = dz + half;
        p.ld[0] = p.ld[1] = ldz;
        p.dh = dh.at[0];
        p.lddh = dh.ld;
        p.padded = true;
        rc = launch_product(p, sms, s);
        p.padded = false;
    }
    p.epi = kStore;
    if (!rc && g.dx) {
        // [dg du] x [Wg Wu]^T: two segments of k, each as long as `hidden`.
        p.x = Factor{{dz, dz + half}, ldz, a.rows, false, {}};
        p.w = Factor{{w.at[0], w.at[1]}, w.ld, a.width, a.w_by_output != 0, {}};
        p.k = a.hidden;
        p.segments = 2;
        p.rows = a.rows;
        p.cols = a.width;
        p.out[0] = g.dx;
        p.ld[0] = g.lddx;
        rc = launch_product(p, sms, s);
        p.segments = 1;
    }
    if (!rc && g.dw) {
        // A product for each half of dw, over the rows of x and of [dg du].
        const Factor z{{dz, dz + half}, ldz, a.hidden, true, {}}, in{{x.at[0], x.at[0]}, x.ld, a.width, true, {}};
        const int64_t es = type_bytes(g.dw_type);
        p.x = a.w_by_output ? z : in;
        p.w = a.w_by_output ? in : z;
        p.k = a.rows;
        p.batch = 2;
        p.beside = g.dx != nullptr;  // dx and dw both come from [dg du], which is there when the kernel of dx begins
        p.rows = p.x.extent;
        p.cols = p.w.extent;
        p.out_type = g.dw_type;
        p.add = g.accumulate != 0;
        p.out[0] = g.dw;
        p.out[1] = static_cast<char*>(g.dw) + (a.w_by_output ? a.hidden * g.lddw : a.hidden) * es;
        p.ld[0] = p.ld[1] = g.lddw;
        rc = launch_product(p, sms, s);
    }
    return rc;
}

int mxfp4_gemm(const mxfp4_gemm_args* args, void* stream)
{
    set_last_error("");
    if (!args)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    const mxfp4_gemm_args& a = *args;
    if (a.rows < 0 || a.cols < 0 || a.width < 0 || a.rows >= kMost || a.cols >= kMost || a.width >= kMost)
        return fail_with(GEMM_ERR_ARG, "sizes must be in [0, 2^31)");
    if (!type_ok(a.out_type))
        return fail_with(GEMM_ERR_ARG, "bad out_type");
    if (a.activation < FFN_NONE || a.activation > FFN_RELU)
        return fail_with(GEMM_ERR_ARG, "unknown activation %d", a.activation);
    if (!a.up_codes && a.activation != FFN_NONE)
        return fail_with(GEMM_ERR_ARG, "an activation needs up_codes");
    if (a.rows == 0 || a.cols == 0)
        return GEMM_OK;
    const int es = type_bytes(a.out_type);
    if (!a.out)
        return fail_with(GEMM_ERR_ARG, "out is NULL");
    if (a.ldo < a.cols || a.ldo >= kMost)
        return fail_with(GEMM_ERR_ARG, "row stride of out below the row, or not below 2^31");
    if (!aligned(a.out, es))
        return fail_with(GEMM_ERR_ALIGN, "out is not aligned to its elements");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.width == 0)
        return cuda_rc(cudaMemset2DAsync(a.out, a.ldo * es, 0, a.cols * es, a.rows, s), "clearing out");
    if (!a.a_codes || !a.a_scales || !a.b_codes || !a.b_scales || (a.up_codes && !a.up_scales))
        return fail_with(GEMM_ERR_ARG, "codes or scales are NULL");
    const int64_t row = ceil_div(a.width, 32) * 16;
    if (a.lda < row || a.ldb < row || (a.up_codes && a.ldu < row) || a.lda >= kMost || a.ldb >= kMost || a.ldu >= kMost)
        return fail_with(GEMM_ERR_ARG, "row stride of codes below the row, or not below 2^31");
    if (!aligned(a.a_codes, 16) || !aligned(a.a_scales, 16) || !aligned(a.b_codes, 16) || !aligned(a.b_scales, 16) ||
        !aligned(a.up_codes, 16) || !aligned(a.up_scales, 16) || a.lda % 16 || a.ldb % 16 || (a.up_codes && a.ldu % 16))
        return fail_with(GEMM_ERR_ALIGN, "codes, their rows and scales must start on 16 bytes");
    int sms = 0;
    const int rc = device_sms(&sms);
    if (rc)
        return rc;
    Product p{};
    p.mx = 1;
    p.epi = a.up_codes ? kGated : kStore;
    p.x = Factor{{a.a_codes, nullptr}, a.lda, a.rows, false, {a.a_scales, nullptr}};
    p.w = Factor{{a.b_codes, a.up_codes}, a.ldb, a.cols, false, {a.b_scales, a.up_scales}, a.ldu};
    p.w_is_weights = true;
    p.k = a.width;
    p.segments = p.batch = 1;
    p.activation = a.activation;
    p.alpha = a.alpha;
    p.out_type = a.out_type;
    p.rows = a.rows;
    p.cols = a.cols;
    p.out[0] = a.out;
    p.ld[0] = a.ldo;
    return launch_product(p, sms, s);
}

}  // extern "C"
