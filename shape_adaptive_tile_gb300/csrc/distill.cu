// Distillation from a teacher's top logits and its gradient (include/rowops.h).
//
// Of many rows a CTA takes one at a time, with two passes over its logits: the
// maximum and the sum of exponentials, and the gradient. The second pass finds
// the row in L2, mostly: the rows at hand in all SMs are 60 MB at most with 128
// threads a CTA, 80 with 256, 120 with 512, and with 1024 as long as 152 rows are
// (159 MB at 262144 tokens in fp32). DRAM reads of a row: 1.0 times at 32768
// tokens in 16-bit types, 1.2 at 131072, 1.14 at 262144. HBM bandwidth bounds it.
//
// Few rows, and the gradient alone, go in slices that lie in shared memory
// while a CTA works on them: fetched by bulk copies (all of a slice in flight
// at once), reduced to a maximum and a sum of exponentials chunk by chunk as
// they land, and, for the gradient, read a second time from there. The CTAs of
// a cluster take a row's slices and put their maxima and sums together through
// distributed shared memory. Slices are cut on 16-byte boundaries of memory,
// wherever the row starts; the ragged ends move by plain loads.
//
// Measured on a GB300, of its copy rate of 6.8 TB/s: 4096 x 131072 bf16 with its
// gradient, an eighth of the rows masked, 361 us (5.58 TB/s, 82%); the loss of
// 1000 x 49999 fp32 36.6 us (81%); the gradient alone of 2047 x 65537 fp16, in
// slices, 86 us (92%); 7 x 32000, in slices, 7.3 us, a chain of latencies.
#include "ptx.cuh"
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kChunk = 16384;       // bytes of a bulk copy with its own barrier
constexpr int kMaxSlice = 65536;    // so that three CTAs' slices fit an SM
constexpr int kMaxChunks = kMaxSlice / kChunk;
constexpr int kMaxCluster = 16;

enum Mode { kLoss, kBoth, kGrad };

// The gradient alone comes from lse, whose rounding to 32 bits is a relative
// error of up to |lse| 2^-24 in q. Rows with more than this (in their logits'
// type, fp32: 4e-6, 16 bits: 3e-5, a sixteenth of fp16's rounding) have their
// sums taken again: rows far from 0, and of the type's lowest value, which have
// nothing of the sum in lse. (us where all rows are, against none: 2047 x 65537
// fp16 180 | 83, 2048 x 65536 fp32 430 | 157, 7 x 131072 bf16 39 | 5.7.)
template <typename T>
constexpr float kFarLse = sizeof(T) == 4 ? 64.0f : 512.0f;

// The teacher's entries of a row in shared memory, four arrays of k rounded up
// to whole 16 bytes, so that the tokens can be compared four at a time.
struct Entries {
    float *p, *log_p, *at_id;  // the teacher's probabilities, their logarithms, the student's logits there (for the loss)
    int* id;                   // -1 for an absent entry, -2 past the last
    int padded;

    static __host__ __device__ constexpr int room(int k) { return (k + 3) / 4 * 16 * 4; }

    __device__ __forceinline__ Entries(void* memory, int k) : padded((k + 3) / 4 * 4)
    {
        p = static_cast<float*>(memory);
        log_p = p + padded, at_id = log_p + padded, id = reinterpret_cast<int*>(at_id + padded);
    }

    // The probability of entry n's token, of all entries that name it, for the first of these; for the others -1.
    __device__ __forceinline__ float of(int n) const
    {
        const int token = id[n];
        float sum = 0.0f;
        for (int l = 0; l < padded; l += 4) {
            const int4 four = *reinterpret_cast<const int4*>(id + l);
            if (four.x != token && four.y != token && four.z != token && four.w != token)
                continue;
            const int names[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (names[e] == token) {
                    if (l + e < n)
                        return -1.0f;
                    sum += p[l + e];
                }
        }
        return sum;
    }
};

// A row's slices, `bytes` each from the 16-byte boundary at or before its
// start. CTA `rank` of the row's `ctas` takes slices rank, rank + ctas, ...
struct Slices {
    int bytes, ctas, per_row;
};

template <typename T>
__device__ __forceinline__ float teacher_at(const void* p, int64_t i)
{
    return to_f32(static_cast<const T*>(p)[i]);
}

__device__ __forceinline__ float teacher_logit(const rowop_distill_args& a, int64_t i)
{
    return a.teacher_type == GEMM_C_F32    ? teacher_at<float>(a.teacher, i)
           : a.teacher_type == GEMM_C_BF16 ? teacher_at<__nv_bfloat16>(a.teacher, i)
                                           : teacher_at<__half>(a.teacher, i);
}

// t (log p - log q) for a student's logit `below` its row's maximum: multiplied
// out, so that neither its quotient by a tiny t nor the square of t leaves fp32.
__device__ __forceinline__ float scaled_log_ratio(const rowop_distill_args& a, float log_p, float below, float log_sum)
{
    return a.temperature * log_p - (below - a.temperature * log_sum);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// The factors of a gradient: of logit v it is share 2^((v - from) scale), less
// the teacher's part.
struct Gradient {
    float share, from, scale;

    __device__ __forceinline__ float of(float v) const { return share * ex2((v - from) * scale); }
};

template <typename T>
__device__ __forceinline__ uint4 gradient_of(const uint4& w, const Gradient& f)
{
    const uint64_t from = pair(-f.from, -f.from), scale = pair(f.scale, f.scale);
    const uint64_t share = pair(f.share, f.share);
    uint64_t v[kPairs<T>];
    unpack_pairs<T>(w, v);
    float o[kPer16<T>];
#pragma unroll
    for (int e = 0; e < kPairs<T>; ++e) {
        const float2 x = halves(mul2(add2(v[e], from), scale));
        const float2 y = halves(mul2(pair(ex2(x.x), ex2(x.y)), share));
        o[2 * e] = y.x, o[2 * e + 1] = y.y;
    }
    return pack16<T>(o);
}

// The gradient of row r by one CTA that takes the row's sums again: a pass over
// the logits in global memory for them, and one for the gradient, which may be
// in the logits' place. `entries` are the row's, `sum` is P, c the factor of the
// whole row. Not inlined, and with few registers: the many rows that never come
// here would pay for them.
template <typename T>
__device__ __noinline__ void gradient_of_far_row(const rowop_distill_args& a, int64_t r, void* entries, Softmax* scratch, float sum, float c,
                                                 float scale)
{
    const Packs<T> s(static_cast<const T*>(a.logits) + r * a.ldl, static_cast<int>(a.vocab));
    T* out = static_cast<T*>(a.dlogits) + r * a.ldd;
    const int k = static_cast<int>(a.k);
    const Entries teacher(entries, k);
    Softmax q = Softmax::none();
#pragma unroll 1
    for (int i = s.inside + threadIdx.x; i < s.end; i += kThreads) {
        const uint4 w[1] = {s.load(i)};
        q.add(softmax_of<T>(w, scale), scale);
    }
    // The elements before and after the whole packs.
    const int before = s.inside ? min(s.element(1), s.vocab) : 0, after = max(s.element(s.end), before);
    auto ends = [&](auto f) {
#pragma unroll 1
    for (int j = threadIdx.x; j < before; j += kThreads)
            f(j);
#pragma unroll 1
    for (int j = after + threadIdx.x; j < s.vocab; j += kThreads)
            f(j);
    };
    ends([&](int j) { q.add(to_f32(s.row[j]), scale); });
#pragma unroll 1
    for (int i = threadIdx.x; i < k; i += kThreads)
        teacher.at_id[i] = teacher.id[i] >= 0 ? to_f32(s.row[teacher.id[i]]) : 0.0f;
    __syncwarp();
    q = cta_softmax<kThreads>(q, scale, scratch);
    const Gradient f = {c * sum / q.sum, q.max, scale};
    if (((reinterpret_cast<uint64_t>(out) ^ reinterpret_cast<uint64_t>(s.row)) & 15) == 0) {
#pragma unroll 1
    for (int i = s.inside + threadIdx.x; i < s.end; i += kThreads)
            *reinterpret_cast<uint4*>(out + s.element(i)) = gradient_of<T>(s.load(i), f);
        ends([&](int j) { out[j] = from_f32<T>(f.of(to_f32(s.row[j]))); });
    } else {
#pragma unroll 1
    for (int j = threadIdx.x; j < s.vocab; j += kThreads)
            out[j] = from_f32<T>(f.of(to_f32(s.row[j])));
    }
    __syncthreads();
#pragma unroll 1
    for (int n = threadIdx.x; n < k; n += kThreads) {
        const float pn = teacher.id[n] >= 0 ? teacher.of(n) : -1.0f;
        if (pn >= 0.0f)
            out[teacher.id[n]] = from_f32<T>(f.of(teacher.at_id[n]) - c * pn);
    }
}

// CTAs an SM that the registers are to allow, for short slices: the gradient
// alone in 16-bit types has 40 (us with | without that bound: 3000 x 5000 22.2 |
// 23.6, 2047 x 65537 77.4 | 78.7, one row of 2048 7.0 | 6.1); the others come to
// 48 by themselves.
template <typename T, int MODE>
constexpr int kSlicePerSM = MODE == kGrad && sizeof(T) == 2 ? 6 : 5;

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, kSlicePerSM<T, MODE> == 6 ? 6 : 0)
    sat_distill_kernel(const __grid_constant__ rowop_distill_args a, const Slices cut)
{
    constexpr int N = kPer16<T>;
    extern __shared__ __align__(128) unsigned char slice[];
    const Entries teacher(slice + cut.bytes, static_cast<int>(a.k));
    float *p = teacher.p, *log_p = teacher.log_p, *at_id = teacher.at_id;
    int* id = teacher.id;
    __shared__ __align__(8) uint64_t bars[kMaxChunks];
    __shared__ Softmax scratch[2][kWarps];
    __shared__ float sums[2 * kWarps];
    __shared__ Softmax across[kMaxCluster];
    const int rank = blockIdx.x % cut.ctas, k = static_cast<int>(a.k);
    const int64_t r = blockIdx.x / cut.ctas;
    const float weight = a.weight ? a.weight[r] : 1.0f;
    const float scale = scale_at(a.temperature);
    const T* row = static_cast<const T*>(a.logits) + r * a.ldl;
    T* out = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ldd : nullptr;
    // The row, and the slices, as addresses.
    const uint64_t start = reinterpret_cast<uint64_t>(row), base = start & ~15ull, stop = start + a.vocab * sizeof(T);
    int phase = 0, packs = 0;
    // This thread has given up a wait; some thread had before the last copies were to start, and they did not.
    bool failed = false, stuck = false;
    int64_t first = 0;  // the element that the slice's first pack starts with (negative where that is before the row)

    // Starts the copies of slice i; every thread then knows its first element and number of packs.
    auto fetch = [&](int i) {
        const uint64_t at = base + static_cast<uint64_t>(i) * cut.bytes;
        const uint64_t lo = at > start ? at : start;
        uint64_t hi = at + cut.bytes < stop ? at + cut.bytes : stop;
        hi = hi > at ? hi : at;  // the last slice may have nothing, as the row may start on any byte of its first 16
        const uint64_t lo16 = (lo + 15) & ~15ull, hi16 = hi & ~15ull;
        first = (static_cast<int64_t>(at) - static_cast<int64_t>(start)) / static_cast<int64_t>(sizeof(T));
        packs = static_cast<int>((hi - at + 15) / 16);
        if (stuck)
            return;
        if (threadIdx.x == 0) {
            for (int c = 0; c < kMaxChunks; ++c) {
                const uint64_t from = at + c * kChunk;
                const uint64_t b = from > lo16 ? from : lo16, e = from + kChunk < hi16 ? from + kChunk : hi16;
                const uint32_t bytes = b < e ? static_cast<uint32_t>(e - b) : 0;
                mbar_arrive_expect_tx(smem_u32(&bars[c]), bytes);
                if (bytes)
                    bulk_load(smem_u32(slice) + static_cast<uint32_t>(b - at), reinterpret_cast<const void*>(b), bytes,
                              smem_u32(&bars[c]));
            }
        }
        // The ends: elements of the packs that are not whole; -inf where there is none.
        if (threadIdx.x >= 32 && threadIdx.x < 32 + 2 * N) {
            const int e = (threadIdx.x - 32) % N;
            const uint64_t pack = threadIdx.x - 32 < N ? lo & ~15ull : hi & ~15ull;
            const uint64_t x = pack + e * sizeof(T);
            const bool whole = pack >= lo && pack + 16 <= hi;
            if (!whole && pack < at + cut.bytes && (threadIdx.x - 32 < N || pack != (lo & ~15ull)))
                *reinterpret_cast<T*>(slice + (x - at)) =
                    x >= lo && x < hi ? *reinterpret_cast<const T*>(x) : from_f32<T>(-INFINITY);
        }
    };
    // Into a slice that has been read, and had its ends written, by ordinary instructions.
    auto refetch = [&](int i) {
        fence_proxy_async_smem();
        stuck = __syncthreads_or(failed);
        fetch(i);
    };
    auto wait = [&](int c) { failed = failed || !wait_bounded<false>(smem_u32(&bars[c]), phase); };
    // Before the CTA ends, where thread 0 has not seen its last copies, of phase `parity`, land.
    auto drain = [&](int parity) {
        for (int c = 0; c < kMaxChunks && threadIdx.x == 0; ++c)
            wait_bounded<false, kDrainNs>(smem_u32(&bars[c]), parity);
    };
    // Writes share 2^((v - from) scale) for the logits v of the slice.
    float share = 0.0f, from = 0.0f;
    auto one_of = [&](float v) { return share * ex2((v - from) * scale); };
    auto write = [&] {
        if (packs == 0)
            return;
        // The packs that lie wholly in the row, 16 bytes each, where the gradient's row starts on the same
        // byte of 16 as the logits'; the rest element by element.
        const bool wide = ((reinterpret_cast<uint64_t>(out) ^ start) & 15) == 0;
        const int begin = !wide ? packs : first < 0 ? 1 : 0;
        const int end = wide && first + static_cast<int64_t>(packs) * N > a.vocab ? packs - 1 : packs;
        const uint64_t from2 = pair(-from, -from), scale2 = pair(scale, scale), share2 = pair(share, share);
        T* to = out + first;
#pragma unroll 4
        for (int i = begin + threadIdx.x; i < end; i += kThreads) {
            uint64_t v[kPairs<T>];
            unpack_pairs<T>(reinterpret_cast<const uint4*>(slice)[i], v);
            float o[N];
#pragma unroll
            for (int e = 0; e < kPairs<T>; ++e) {
                const float2 x = halves(mul2(add2(v[e], from2), scale2));
                const float2 y = halves(mul2(pair(ex2(x.x), ex2(x.y)), share2));
                o[2 * e] = y.x, o[2 * e + 1] = y.y;
            }
            *reinterpret_cast<uint4*>(to + static_cast<int64_t>(i) * N) = pack16<T>(o);
        }
        auto one = [&](int j) {
            if (first + j >= 0 && first + j < a.vocab)
                to[j] = from_f32<T>(one_of(to_f32(reinterpret_cast<const T*>(slice)[j])));
        };
        if (!wide)
            for (int j = threadIdx.x; j < packs * N; j += kThreads)
                one(j);
        else if (threadIdx.x < N && begin == 1)
            one(threadIdx.x);
        if (wide && threadIdx.x >= 32 && threadIdx.x < 32 + N && end < packs && (end > 0 || begin == 0))
            one(end * N + threadIdx.x - 32);
    };
    auto write_zeros = [&] {
        for (int64_t j = rank * static_cast<int64_t>(kThreads) + threadIdx.x; j < a.vocab; j += cut.ctas * kThreads)
            out[j] = from_f32<T>(0.0f);
    };

    // A thread's first entry, on its way with the weight.
    const bool entry = (MODE != kLoss || rank == 0) && threadIdx.x < k;
    const int token0 = entry ? a.ids[r * a.ldi + threadIdx.x] : -1;
    const float logit0 = entry ? teacher_logit(a, r * a.ldt + threadIdx.x) : 0.0f;
    const float lse = MODE == kGrad ? a.lse[r] : 0.0f;
    if (weight == 0.0f) {  // alike for all CTAs of the cluster
        if (MODE != kGrad && rank == 0 && threadIdx.x == 0) {
            a.loss[r] = 0.0f;
            if (a.lse)
                a.lse[r] = 0.0f;
        }
        if (MODE != kLoss)
            write_zeros();
        return;
    }
    if (threadIdx.x == 0) {
        for (int c = 0; c < kMaxChunks; ++c)
            mbar_init(smem_u32(&bars[c]), 1);
        fence_mbar_init();
    }
    __syncthreads();
    const bool any = rank < cut.per_row;
    if (any)
        fetch(rank);
    __syncwarp();
    if (MODE != kGrad && cut.ctas > 1)
        cluster_arrive();  // waited for before the first store to another CTA, which has to have started by then

    // The teacher's entries, while the first slice is on its way.
    bool empty = false;
    float sum[1] = {0.0f};
    int turn = 0;
    if (MODE != kLoss || rank == 0) {
        Softmax t = Softmax::none();
        if (threadIdx.x < teacher.padded - k)
            id[k + threadIdx.x] = -2;
        for (int i = threadIdx.x; i < k; i += kThreads) {
            const bool held = i == static_cast<int>(threadIdx.x);
            const int token = held ? token0 : a.ids[r * a.ldi + i];
            const float v = held ? logit0 : teacher_logit(a, r * a.ldt + i);
            const bool there = token >= 0 && token < a.vocab && v != -INFINITY;
            id[i] = there ? token : -1;
            log_p[i] = v;
            // Before any CTA of the cluster writes its part of the gradient, which may be in the logits' place.
            if (MODE != kGrad && rank == 0)
                at_id[i] = there ? to_f32(row[token]) : 0.0f;
            if (there)
                t.add(v, scale);
        }
        t = cta_softmax<kThreads>(t, scale, scratch[0]);
        empty = t.max == -INFINITY && t.sum == 0.0f;  // entries of NaN are present: they are in the sum
        const float top = a.teacher_lse ? 0.0f : t.max, rest = a.teacher_lse ? a.teacher_lse[r] : logf(t.sum);
        for (int i = threadIdx.x; i < k; i += kThreads) {
            log_p[i] = (log_p[i] - top) / a.temperature - rest;
            p[i] = id[i] >= 0 ? expf(log_p[i]) : 0.0f;
            sum[0] += p[i];
        }
        row_sums<kThreads>(sum, sums, turn);
    }

    auto factor = [&] { return (a.dloss ? a.dloss[r] : 1.0f) * weight * a.temperature; };
    if (MODE == kGrad && (empty || fabsf(lse) > kFarLse<T>)) {
        if (any)  // the copies have to land before the CTA ends
            drain(phase);
        if (empty)
            write_zeros();
        else if (rank == 0)
            gradient_of_far_row<T>(a, r, slice + cut.bytes, scratch[1], sum[0], factor(), scale);
        return;
    }
    Softmax q = Softmax::none();
    if (MODE != kGrad) {
        for (int i = rank; i < cut.per_row; i += cut.ctas) {
            if (i != rank)
                refetch(i);
            __syncthreads();  // the ends are written
            if (stuck)
                break;
            for (int c = 0; c < kMaxChunks; ++c) {
                wait(c);
                const int end = min(packs, (c + 1) * (kChunk / 16));
                const int begin = c * (kChunk / 16) + threadIdx.x;
                constexpr int U = kChunk / 16 / kThreads;
                if (begin < end) {
                    uint4 w[U];
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        w[u] = begin + u * kThreads < end ? reinterpret_cast<const uint4*>(slice)[begin + u * kThreads] : nothing<T>();
                    q.add(softmax_of<T>(w, scale), scale);
                }
            }
            phase ^= 1;
        }
        if (failed || stuck)
            q.sum = NAN;
        q = cta_softmax<kThreads>(q, scale, scratch[1]);
        if (cut.ctas > 1) {
            cluster_wait();
            if (threadIdx.x < cut.ctas) {
                const uint32_t at = map_to_cta(smem_u32(&across[rank]), threadIdx.x);
                st_cluster_f32(at, q.max);
                st_cluster_f32(at + 4, q.sum);
            }
            __syncwarp();
            cluster_sync();
            q = sum_softmax(across, 1, cut.ctas, scale);
        }
        const float log_sum = logf(q.sum);
        if (rank == 0) {
            float loss[1] = {0.0f};
            for (int i = threadIdx.x; i < k; i += kThreads)
                if (p[i] != 0.0f)
                    loss[0] += p[i] * scaled_log_ratio(a, log_p[i], at_id[i] - q.max, log_sum);
            row_sums<kThreads>(loss, sums, turn);
            if (threadIdx.x == 0) {
                a.loss[r] = empty ? 0.0f : weight * a.temperature * loss[0];
                if (a.lse)
                    a.lse[r] = empty ? 0.0f : q.max / a.temperature + log_sum;
            }
        }
    }
    if (MODE == kLoss || empty) {
        if (failed)
            drain(phase ^ 1);
        if (MODE != kLoss)
            write_zeros();
        return;
    }
    const float c = factor();
    if (MODE == kGrad) {
        share = c * sum[0], from = lse * a.temperature;
    } else {
        share = c * sum[0] / q.sum, from = q.max;
    }
    const bool resident = MODE == kBoth && cut.per_row <= cut.ctas;
    for (int i = rank; i < cut.per_row; i += cut.ctas) {
        if (!resident) {
            if (MODE == kBoth || i != rank)
                refetch(i);
            __syncthreads();
            for (int n = 0; n < kMaxChunks && !stuck; ++n)
                wait(n);
            phase ^= !stuck;
            if (failed || stuck)
                share = NAN;
        }
        write();
        __syncthreads();
        // The teacher's tokens within the slice, each once: by the first of the entries that name it.
        const int64_t last = min(first + static_cast<int64_t>(packs) * N, a.vocab);
        for (int n = threadIdx.x; n < k; n += kThreads) {
            if (id[n] < max(first, int64_t{0}) || id[n] >= last)
                continue;
            const float pn = teacher.of(n);
            if (pn >= 0.0f) {
                const float v = to_f32(reinterpret_cast<const T*>(slice)[id[n] - first]);
                out[id[n]] = from_f32<T>(one_of(v) - c * pn);
            }
        }
    }
    if (failed)
        drain(phase ^ 1);
}

// ---- many rows: a CTA a row -----------------------------------------------------

constexpr int64_t kSMs = 152, kSmemPerSM = 227 * 1024;

// Sixteen bytes by a load that tells L2 how long to keep them.
__device__ __forceinline__ uint4 load_hinted(const void* p, uint64_t policy)
{
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.b32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}

template <typename T, int MODE, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) sat_distill_row_kernel(const __grid_constant__ rowop_distill_args a)
{
    constexpr int N = kPer16<T>, U = 8, W = NT / 32;
    extern __shared__ __align__(16) unsigned char entries[];
    __shared__ Softmax scratch[2][W];
    __shared__ float sums[2 * W];
    const int k = static_cast<int>(a.k), vocab = static_cast<int>(a.vocab), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Entries teacher(entries, k);
    float *p = teacher.p, *log_p = teacher.log_p, *at_id = teacher.at_id;
    int* id = teacher.id;
    const int64_t r = blockIdx.x;
    const float weight = a.weight ? a.weight[r] : 1.0f, scale = scale_at(a.temperature);
    const Packs<T> s(static_cast<const T*>(a.logits) + r * a.ldl, vocab);
    T* out = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ldd : nullptr;
    int turn = 0;

    // f(packs, first, all) for the row's packs in batches of U a thread, all of a batch's loads first; packs past the end are -inf.
    auto batches = [&](uint64_t policy, auto f) {
        auto load = [&](int j) { return load_hinted(s.row + s.element(j), policy); };
        int j = s.inside + threadIdx.x;
        for (; j - static_cast<int>(threadIdx.x) + U * NT <= s.end; j += U * NT) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = load(j + u * NT);
            f(w, j, true);
        }
        if (j < s.end) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = j + u * NT < s.end ? load(j + u * NT) : nothing<T>();
            f(w, j, false);
        }
    };
    // The first pass's lines are to stay in L2 for the second, after which they are of no more use.
    uint64_t keep, drop;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(drop));
    // The column of the element at the row's ends, outside whole packs, that this lane of the last warp sees to.
    const int end_column = warp < W - 1 || lane >= 2 * N ? -1
                           : lane < N                            ? (s.inside ? lane - s.shift : -1)
                                                                 : s.element(s.end) + lane - N;
    const bool at_end = end_column >= 0 && end_column < vocab;

    Softmax t = Softmax::none();
    if (threadIdx.x < teacher.padded - k)
        id[k + threadIdx.x] = -2;
    if (weight != 0.0f)
        for (int i = threadIdx.x; i < k; i += NT) {
            const int token = a.ids[r * a.ldi + i];
            const float v = teacher_logit(a, r * a.ldt + i);
            const bool there = token >= 0 && token < vocab && v != -INFINITY;
            id[i] = there ? token : -1;
            log_p[i] = v;
            at_id[i] = there ? to_f32(s.row[token]) : 0.0f;  // before the gradient, which may be in the logits' place
            if (there)
                t.add(v, scale);
        }
    t = cta_softmax<NT>(t, scale, scratch[0]);
    if (t.max == -INFINITY && t.sum == 0.0f) {  // masked, or no entry present (those of NaN are in the sum)
        if (threadIdx.x == 0) {
            a.loss[r] = 0.0f;
            if (a.lse)
                a.lse[r] = 0.0f;
        }
        if (MODE == kBoth) {
            const Packs<T> o(out, vocab);
            for (int j = o.inside + threadIdx.x; j < o.end; j += NT)
                *reinterpret_cast<uint4*>(out + o.element(j)) = make_uint4(0, 0, 0, 0);
            if (warp == W - 1 && lane < 2 * N) {
                const int c = lane < N ? (o.inside ? lane - o.shift : -1) : o.element(o.end) + lane - N;
                if (c >= 0 && c < vocab)
                    out[c] = from_f32<T>(0.0f);
            }
        }
        return;
    }
    const float top = a.teacher_lse ? 0.0f : t.max, rest = a.teacher_lse ? a.teacher_lse[r] : logf(t.sum);

    Softmax q = Softmax::none();
    batches(MODE == kBoth ? keep : drop, [&](const uint4(&w)[U], int, bool) { q.add(softmax_of<T>(w, scale), scale); });
    if (at_end)
        q.add(to_f32(s.row[end_column]), scale);
    __syncwarp();
    q = cta_softmax<NT>(q, scale, scratch[1]);
    const float log_sum = logf(q.sum);
    float sum[2] = {0.0f, 0.0f};  // of p, and of p (log p - log q)
    for (int i = threadIdx.x; i < k; i += NT) {
        log_p[i] = (log_p[i] - top) / a.temperature - rest;
        p[i] = id[i] >= 0 ? expf(log_p[i]) : 0.0f;
        sum[0] += p[i];
        if (p[i] != 0.0f)
            sum[1] += p[i] * scaled_log_ratio(a, log_p[i], at_id[i] - q.max, log_sum);
    }
    row_sums<NT>(sum, sums, turn);
    if (threadIdx.x == 0) {
        a.loss[r] = weight * a.temperature * sum[1];
        if (a.lse)
            a.lse[r] = q.max / a.temperature + log_sum;
    }
    if (MODE == kLoss)
        return;
    const float c = (a.dloss ? a.dloss[r] : 1.0f) * weight * a.temperature;
    const Gradient f = {c * sum[0] / q.sum, q.max, scale};
    if (((reinterpret_cast<uint64_t>(out) ^ reinterpret_cast<uint64_t>(s.row)) & 15) == 0) {
        batches(drop, [&](const uint4(&w)[U], int j, bool all) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (all || j + u * NT < s.end)
                    __stcs(reinterpret_cast<uint4*>(out + s.element(j + u * NT)), gradient_of<T>(w[u], f));
        });
        if (at_end)
            out[end_column] = from_f32<T>(f.of(to_f32(s.row[end_column])));
    } else {  // rows that begin on other bytes of 16 than the logits': element by element
        for (int j = threadIdx.x; j < vocab; j += NT)
            out[j] = from_f32<T>(f.of(to_f32(s.row[j])));
    }
    __syncthreads();
    // The teacher's tokens, each once: by the first of the entries that name it.
    for (int n = threadIdx.x; n < k; n += NT) {
        if (id[n] < 0)
            continue;
        const float pn = teacher.of(n);
        if (pn >= 0.0f)
            out[id[n]] = from_f32<T>(f.of(at_id[n]) - c * pn);
    }
}

int check(const rowop_distill_args* a, bool forward)
{
    if (!a)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    if (a->rows < 0 || a->vocab < 0 || a->k < 0)
        return fail_with(GEMM_ERR_ARG, "negative size");
    if (a->rows == 0)
        return GEMM_OK;
    if (a->rows > (1 << 26))
        return fail_with(GEMM_ERR_ARG, "rows %lld is above 2^26", (long long)a->rows);
    if (a->vocab < 1 || a->vocab > (INT64_C(1) << 30))
        return fail_with(GEMM_ERR_ARG, "vocab %lld is not within 1 .. 2^30", (long long)a->vocab);
    if (a->k > ROWOP_DISTILL_MAX_K)
        return fail_with(GEMM_ERR_ARG, "k %lld is above %d", (long long)a->k, ROWOP_DISTILL_MAX_K);
    if (!type_ok(a->logits_type) || !type_ok(a->teacher_type))
        return fail_with(GEMM_ERR_ARG, "bad type");
    if (!(a->temperature > 0.0f) || a->temperature > 3e38f)
        return fail_with(GEMM_ERR_ARG, "temperature must be finite and above 0");
    if (!a->logits || (a->k > 0 && (!a->ids || !a->teacher)))
        return fail_with(GEMM_ERR_ARG, "logits, ids or teacher is NULL");
    if (forward ? !a->loss : !a->lse || !a->dlogits)
        return fail_with(GEMM_ERR_ARG, forward ? "loss is NULL" : "lse or dlogits is NULL");
    if (a->ldl < a->vocab || (a->dlogits && a->ldd < a->vocab) || (a->k > 0 && (a->ldi < a->k || a->ldt < a->k)))
        return fail_with(GEMM_ERR_ARG, "row stride below the row's length");
    if (!aligned(a->logits, type_bytes(a->logits_type)) || !aligned(a->dlogits, type_bytes(a->logits_type)) ||
        !aligned(a->teacher, type_bytes(a->teacher_type)) || !aligned(a->ids, 4) || !aligned(a->teacher_lse, 4) ||
        !aligned(a->weight, 4) || !aligned(a->loss, 4) || !aligned(a->lse, 4) || !aligned(a->dloss, 4))
        return fail_with(GEMM_ERR_ALIGN, "a pointer is not aligned to its elements");
    return GEMM_OK;
}

template <typename T, int MODE, int NT>
cudaError_t launch_rows_by(const rowop_distill_args& a, cudaStream_t s)
{
    sat_distill_row_kernel<T, MODE, NT><<<static_cast<unsigned>(a.rows), NT, Entries::room(static_cast<int>(a.k)), s>>>(a);
    return cudaGetLastError();
}

// The threads of a row's CTA, and with them the rows at hand in an SM (1024 /
// NT): more of these overlap better, but with a gradient the rows at hand
// should be in L2 for their second pass. (us for 128 | 256 | 512 | 1024 threads,
// with gradient: 1500 rows in 16-bit types of 24576 tokens 38 | 42 | 54 | 104,
// 49152 72 | 62 | 77 | 118, 131072 200 | 172 | 152 | 182, 700 x 262144 179 | 197 |
// 168 | 155; fp32 1500 x 24576 71 | 59 | 71 | 112, 700 x 131072 178 | 193 | 166 |
// 150, 400 x 262144 206 | 204 | 206 | 184. Loss: 1500 x 32768 22 | 23 | 29 | 59,
// 131072 68 | 65 | 67 | 84; 700 x 262144, one round of eight CTAs an SM and 1.2 of
// four, 58 | 69 | 66 | 68.)
template <typename T, int MODE>
cudaError_t launch_rows(const rowop_distill_args& a, int64_t row, cudaStream_t s)
{
    if (row <= (MODE == kLoss ? 131072 : 49152))
        return launch_rows_by<T, MODE, 128>(a, s);
    if (MODE == kLoss || row <= 131072)
        return launch_rows_by<T, MODE, 256>(a, s);
    if constexpr (MODE == kBoth)
        return row <= 393216 ? launch_rows_by<T, MODE, 512>(a, s) : launch_rows_by<T, MODE, 1024>(a, s);
    return cudaErrorInvalidValue;
}

template <typename T, int MODE>
cudaError_t launch(const rowop_distill_args& a, cudaStream_t s)
{
    // With what a row may need before its start to reach a 16-byte boundary.
    const bool even = aligned(a.logits, 16) && a.ldl * sizeof(T) % 16 == 0;
    const int64_t bytes = a.vocab * static_cast<int64_t>(sizeof(T)) + (even ? 0 : 15);
    // Slices of a cluster's CTAs: of 64 KB at most, so that three CTAs share an
    // SM and one's copies overlap another's arithmetic; smaller, down to 4 KB,
    // where there are too few rows to fill the GPU with two CTAs per SM.
    Slices cut;
    cut.ctas = 1;
    while (cut.ctas < kMaxCluster && (bytes > static_cast<int64_t>(cut.ctas) * kMaxSlice ||
                                      (a.rows * cut.ctas < 304 && bytes > static_cast<int64_t>(cut.ctas) * 4096)))
        cut.ctas *= 2;
    const int64_t each = (bytes + cut.ctas - 1) / cut.ctas;
    cut.bytes = static_cast<int>(each < kMaxSlice ? (each + 127) / 128 * 128 : kMaxSlice);
    cut.per_row = static_cast<int>((bytes + cut.bytes - 1) / cut.bytes);
    const int smem = cut.bytes + Entries::room(static_cast<int>(a.k));
    if constexpr (MODE != kGrad) {
        // A CTA a row, or a row's slices in a cluster: a row by itself where it is short, where there are rows for two thirds
        // of the SMs, and from half of them on where the clusters do not all run at once. (us, row | slices, with gradient:
        // bf16 8 x 16384 7.7 | 7.7, 8 x 32000 8.8 | 8.1, 88 x 32000 11.2 | 11.3, 8 x 131072 17.9 | 9.6, 100 x 131072 20.5 |
        // 19.5, 114 x 131072 20.5 | 28.2, 304 x 131072 36 | 50; fp32 76 x 102336 24.1 | 19.2 (608 CTAs of 50 KB, four an SM),
        // 88 x 102336 24.7 | 26.9, 64 x 262144 43.2 | 44.9, 76 x 262144 45.7 | 55.8. Loss: bf16 38 x 32000 7.2 | 7.6, 76 x 50304
        // 10.0 | 8.4, 100 x 131072 12.6 | 12.6, 114 x 131072 12.7 | 17.3; fp32 64 x 262144 30.3 | 25.1, 76 x 262144 30.6 | 31.1.)
        const int64_t row = a.vocab * static_cast<int64_t>(sizeof(T));
        const int64_t fit = kSmemPerSM / (smem + 2048), at_once = kSMs * (fit < kSlicePerSM<T, MODE> ? fit : kSlicePerSM<T, MODE>);
        if (row <= (MODE == kLoss ? 65536 : 32768) || 3 * a.rows >= 2 * kSMs || (2 * a.rows >= kSMs && a.rows * cut.ctas > at_once))
            return launch_rows<T, MODE>(a, row, s);
    }
    auto kernel = sat_distill_kernel<T, MODE>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel), kMaxSlice + Entries::room(ROWOP_DISTILL_MAX_K));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = MODE == kGrad ? 1 : static_cast<unsigned>(cut.ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * cut.ctas));
    return cudaLaunchKernelEx(&cfg, kernel, a, cut);
}

template <int MODE>
int run(const rowop_distill_args& a, cudaStream_t s)
{
    const cudaError_t e = a.logits_type == GEMM_C_F32    ? launch<float, MODE>(a, s)
                          : a.logits_type == GEMM_C_BF16 ? launch<__nv_bfloat16, MODE>(a, s)
                                                         : launch<__half, MODE>(a, s);
    return e == cudaSuccess ? GEMM_OK
                            : fail_with(GEMM_ERR_LAUNCH, "launching the distillation kernel: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int rowop_distill(const rowop_distill_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args, true);
    if (rc || args->rows == 0)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return args->dlogits ? run<kBoth>(*args, s) : run<kLoss>(*args, s);
}

int rowop_distill_backward(const rowop_distill_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args, false);
    if (rc || args->rows == 0)
        return rc;
    return run<kGrad>(*args, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
