// Verification of drafted tokens and the draw of the next one (include/rowops.h).
//
// Two kernels. The first reads every row of every sequence once: each warp
// takes its share of the rows' parts, 4 KB in 16-bit types and all of them in
// flight at once, and leaves a part's maximum and sum of exponentials in the
// workspace; HBM bandwidth bounds it. In the second several CTAs take a
// sequence: each puts the parts together, all decide alike which token is the
// first refused, and each races through its share of that one row (from L2,
// mostly, and the noise with it, which the first kernel had fetched there). The
// last of them to finish has the winner. The second kernel's CTAs start while
// the first one's last ones run.
//
// Measured on a GB300: 64 x 5 drafts of 131072 tokens in bf16 39 us, of which the
// first kernel 23 (134 MB, 70% of the DRAM rate) and the race most of the rest:
// its loads' latency bounds it. 193 x 3 of 65537 in fp16 39 us; 1 x 4 of 32768
// 10 us, a chain of two kernels' latencies. One kernel with a cluster a sequence
// took 55 us for the first of these, a CTA a part of a row 56.
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxRows = 2 * ROWOP_VERIFY_MAX_DRAFTS + 1;

// What is kept of a row (or of a part or a warp's share of it): its softmax,
// and for the greedy choice its largest value's lowest token.
struct __align__(16) RowStats {
    Softmax q;
    float value;
    int best;
};

// The larger value, or of equals the lower index; an index of -1 is none.
__device__ __forceinline__ void take(float& v, int& at, float v2, int at2)
{
    if (at2 >= 0 && (at < 0 || v2 > v || (v2 == v && at2 < at)))
        v = v2, at = at2;
}

__device__ __forceinline__ void warp_best(float& v, int& at)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(v, at, __shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, at, o));
}

// N consecutive elements from row[j] on, of a row of `vocab`: by 16-byte loads
// from the boundary before them, shifted into place, where all that these
// touch lies in the row. The shift is the same for all lanes.
template <int N, typename T>
__device__ __forceinline__ void load_window(float (&v)[N], const T* row, int j, int vocab)
{
    constexpr int V = N / kPer16<T>, P = kPer16<T>;
    const int shift = static_cast<int>((reinterpret_cast<uint64_t>(row + j) & 15) / sizeof(T));
    const int first = j - shift;
    if (shift == 0 || (first >= 0 && first + (V + 1) * P <= vocab)) {
        uint32_t w[4 * V + 4];
#pragma unroll
        for (int h = 0; h <= V; ++h)
            if (h < V || shift) {
                const uint4 x = *reinterpret_cast<const uint4*>(row + first + h * P);
                w[4 * h] = x.x, w[4 * h + 1] = x.y, w[4 * h + 2] = x.z, w[4 * h + 3] = x.w;
            }
        const int words = shift * static_cast<int>(sizeof(T)) / 4;
        if (words & 2)
#pragma unroll
            for (int k = 0; k < 4 * V + 2; ++k)
                w[k] = w[k + 2];
        if (words & 1)
#pragma unroll
            for (int k = 0; k < 4 * V + 1; ++k)
                w[k] = w[k + 1];
        if constexpr (sizeof(T) == 2) {
            if (shift & 1)
#pragma unroll
                for (int k = 0; k < 4 * V; ++k)
                    w[k] = __funnelshift_r(w[k], w[k + 1], 16);
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
                const float2 f = unpack2<T>(w[k]);
                v[2 * k] = f.x, v[2 * k + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                v[k] = __uint_as_float(w[k]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = to_f32(row[j + e]);
    }
}

// The same where that is a boundary.
template <int N, typename T>
__device__ __forceinline__ void load_beside(float (&v)[N], const T* row, int j)
{
#pragma unroll
    for (int h = 0; h < N / kPer16<T>; ++h) {
        float u[kPer16<T>];
        unpack16<T>(*reinterpret_cast<const uint4*>(row + j + h * kPer16<T>), u);
#pragma unroll
        for (int e = 0; e < kPer16<T>; ++e)
            v[h * kPer16<T> + e] = u[e];
    }
}

// The rows' parts: `elements` of a row each.
struct Parts {
    int elements, per_row;
};

constexpr int kCtas = 4 * 152;     // of the first kernel: four an SM
constexpr int kMaxScan = 1024;     // sequences whose lengths its CTAs add up

Parts parts_of(int64_t batch, int64_t drafts, int64_t vocab)
{
    // 2048 elements, 64 a lane; fewer, down to 512, where two warps an SM's
    // scheduler would not come of it; more where a row would have over 512.
    const int64_t rows = batch * (2 * drafts + 1);
    int64_t each = 2048;
    // A row may start up to 7 elements after a 16-byte boundary.
    auto count = [&] { return (vocab + 7 + each - 1) / each; };
    while (each > 512 && rows * count() < 8 * 152)
        each /= 2;
    while (count() > 512 || rows * count() > (1 << 30))
        each *= 2;
    return {static_cast<int>(each), static_cast<int>(count())};
}

// CTAs of the second kernel for a sequence: four an SM in all, of at least
// 2048 elements of the race each.
int racers_of(int64_t batch, int64_t vocab)
{
    const int64_t fit = 4 * 152 / batch, want = (vocab + 2047) / 2048, n = fit < want ? fit : want;
    return static_cast<int>(n < 1 ? 1 : n < 64 ? n : 64);
}

// What the second kernel's CTAs of a sequence leave for the last of them.
constexpr int kMaxRacers = 64;

struct __align__(16) Races {
    float value[kMaxRacers];
    int token[kMaxRacers];
    unsigned done;
};

// Behind the parts in the workspace.
__device__ __forceinline__ Races* races_of(const rowop_verify_args& a, const Parts& parts)
{
    return reinterpret_cast<Races*>(static_cast<RowStats*>(a.workspace) + a.batch * (2 * a.drafts + 1) * parts.per_row);
}

__device__ __forceinline__ int length_of(const rowop_verify_args& a, int64_t b)
{
    const int drafts = static_cast<int>(a.drafts);
    return a.lengths ? min(max(a.lengths[b], 0), drafts) : drafts;
}

// Scales of the exponents: a greedy target's log probabilities are at temperature 1.
template <bool kGreedy>
__device__ __forceinline__ float target_scale(const rowop_verify_args& a)
{
    return kGreedy ? kLog2e : scale_at(a.temperature);
}

// All sequences' rows in order (of each the target's 0 .. length, then the
// draft's 0 .. length - 1) have their parts dealt to the grid's warps in equal
// runs. The rows before each sequence are counted by every CTA for itself;
// past kMaxScan sequences, all `drafts` rows are counted and those past the
// lengths skipped.
template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kThreads, 4)
    sat_verify_rows_kernel(const __grid_constant__ rowop_verify_args a, const Parts parts)
{
    constexpr int N = kPer16<T>, U = 8;
    __shared__ int before[kMaxScan + 1], sums[kWarps];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int drafts = static_cast<int>(a.drafts), vocab = static_cast<int>(a.vocab), batch = static_cast<int>(a.batch);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool point = kGreedy || !a.draft, scan = a.lengths && batch <= kMaxScan;
    const int most = drafts + 1 + (point ? 0 : drafts);
    auto rows_for = [&](int len) { return len + 1 + (point ? 0 : len); };
    int total = batch * most;
    if (scan) {
        constexpr int S = kMaxScan / kThreads;
        int n[S], sum = 0;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int b = threadIdx.x * S + i;
            n[i] = b < batch ? rows_for(length_of(a, b)) : 0;
            sum += n[i];
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? v : 0;
        }
        if (lane == 31)
            sums[warp] = upto;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            upto += sums[w];
        int at = upto - sum;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            before[threadIdx.x * S + i] = at;
            at += n[i];
        }
        if (threadIdx.x == kThreads - 1)
            before[kMaxScan] = at;
        __syncthreads();
        total = before[kMaxScan];
    }
    // This warp's run of parts, and the sequence, row and part that it begins with.
    const int warps = gridDim.x * kWarps, me = blockIdx.x * kWarps + warp;
    const int64_t items = static_cast<int64_t>(total) * parts.per_row;
    int item = static_cast<int>(items * me / warps);
    const int stop = static_cast<int>(items * (me + 1) / warps);
    if (item >= stop)
        return;
    const int first_row = item / parts.per_row;
    int part = item - first_row * parts.per_row, b, i;
    if (scan) {
        int low = 0, high = batch - 1;  // the last sequence with no more rows before it
        while (low < high) {
            const int mid = (low + high + 1) / 2;
            if (before[mid] <= first_row)
                low = mid;
            else
                high = mid - 1;
        }
        b = low, i = first_row - before[b];
    } else {
        b = first_row / most, i = first_row - b * most;
    }
    int len = length_of(a, b);
    for (int more; item < stop; item += more, part = 0, ++i) {
        more = min(parts.per_row - part, stop - item);  // this row's parts of the run, taken as one
        if (i == (scan ? rows_for(len) : most))
            i = 0, len = length_of(a, ++b);
        // Past the scan the target's rows are drafts + 1 always.
        const int targets = scan ? len + 1 : drafts + 1;
        const bool target = i < targets;
        const int r = target ? i : i - targets;
        if (!scan && (target ? r > len : r >= len))
            continue;
        const Packs<T> s(target ? static_cast<const T*>(a.target) + (static_cast<int64_t>(b) * (drafts + 1) + r) * a.ldt
                                : static_cast<const T*>(a.draft) + (static_cast<int64_t>(b) * drafts + r) * a.ldq, vocab);
        const float scale = target ? target_scale<kGreedy>(a) : scale_at(a.draft_temperature);
        const int first = part * (parts.elements / N), last = min(first + more * (parts.elements / N), s.count);
        const int begin = max(first, s.inside), end = min(last, s.end);
        RowStats st = {Softmax::none(), -INFINITY, -1};
        int top_batch = 0;  // the first batch that has the largest value
        auto add = [&](const uint4(&w)[U], int j) {
            const Softmax q = softmax_of<T>(w, scale);
            if (kGreedy && q.max > st.value)
                st.value = q.max, top_batch = j;
            st.q.add(q, scale);
        };
        int j = begin + lane;
        for (const uint4* at = reinterpret_cast<const uint4*>(s.row + s.element(j)); j - lane + U * 32 <= end; j += U * 32, at += U * 32) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = at[u * 32];
            add(w, j);
        }
        if (j - lane < end) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = j + u * 32 < end ? s.load(j + u * 32) : nothing<T>();
            add(w, j);
        }
        if (kGreedy && st.value > -INFINITY)  // its lowest token: the batch again
#pragma unroll 1
            for (int u = 0; u < U && st.best < 0; ++u) {
                float v[N];
                unpack16<T>(top_batch + u * 32 < end ? s.load(top_batch + u * 32) : nothing<T>(), v);
#pragma unroll
                for (int e = N - 1; e >= 0; --e)
                    st.best = v[e] == st.value ? s.element(top_batch + u * 32) + e : st.best;
            }
        // The packs at the row's ends, an element a lane.
        if (lane < 2 * N) {
            const int c = lane < N ? (s.inside && part == 0 ? lane - s.shift : -1)
                                   : s.end < last && s.end >= first ? s.element(s.end) + lane - N : -1;
            if (c >= 0 && c < vocab) {
                const float v = to_f32(s.row[c]);
                if (kGreedy && v > -INFINITY)
                    take(st.value, st.best, v, c);
                st.q.add(v, scale);
            }
        }
        __syncwarp();
        st.q = warp_softmax(st.q, scale);
        if (kGreedy)
            warp_best(st.value, st.best);
        // All of the run in the first part's place, nothing in the others'.
        RowStats* to = static_cast<RowStats*>(a.workspace) +
                       (static_cast<int64_t>(b) * (2 * drafts + 1) + (target ? r : drafts + 1 + r)) * parts.per_row + part;
        for (int c = lane; c < more; c += 32)
            to[c] = c == 0 ? st : RowStats{Softmax::none(), -INFINITY, -1};
        // The sequence's CTAs of the second kernel count themselves from 0.
        if (i == 0 && part == 0 && lane == 0)
            races_of(a, parts)[b].done = 0;
        // The noise that the sequence's draw will want, towards L2.
        if (!kGreedy && i == 0) {
            const char* noise = reinterpret_cast<const char*>(a.noise + b * a.ldn);
            const int64_t to = min((part + more) * static_cast<int64_t>(parts.elements), a.vocab) * 4;
            for (int64_t at = part * static_cast<int64_t>(parts.elements) * 4 + lane * 128; at < to; at += 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + at));
        }
    }
}

// `ctas` CTAs a sequence: the decisions, then the draw.
template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kThreads, 4)
    sat_verify_draw_kernel(const __grid_constant__ rowop_verify_args a, const Parts parts, int ctas)
{
    constexpr int N = kPer16<T>;
    __shared__ RowStats whole[kMaxRows];  // of the target's rows, then the draft's
    __shared__ float logit[2][ROWOP_VERIFY_MAX_DRAFTS];  // the target's and the draft's at the drafted tokens
    __shared__ float values[kWarps];
    __shared__ int where[kWarps];
    __shared__ int refused;
    __shared__ bool last;
    const int rank = blockIdx.x % ctas, drafts = static_cast<int>(a.drafts), vocab = static_cast<int>(a.vocab);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t b = blockIdx.x / ctas;
    const int len = length_of(a, b);
    const bool point = kGreedy || !a.draft;
    const float scale = target_scale<kGreedy>(a), q_scale = point ? 0.0f : scale_at(a.draft_temperature);
    const int rows = len + 1 + (point ? 0 : len);
    auto target_row = [&](int i) { return static_cast<const T*>(a.target) + (b * (drafts + 1) + i) * a.ldt; };
    auto draft_row = [&](int i) { return static_cast<const T*>(a.draft) + (b * drafts + i) * a.ldq; };
    if (threadIdx.x < len) {
        const int i = threadIdx.x, token = a.tokens[b * drafts + i];
        const bool there = token >= 0 && token < vocab;
        logit[0][i] = there ? to_f32(target_row(i)[token]) : -INFINITY;
        logit[1][i] = there && !point ? to_f32(draft_row(i)[token]) : 0.0f;
    }
    if (threadIdx.x == 0)
        refused = len;
    // What the first kernel left, a warp a row: lanes, then the lanes' sums in order.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = warp; i < rows; i += kWarps) {
        const float by = i <= len ? scale : q_scale;
        const int64_t row = b * (2 * drafts + 1) + (i <= len ? i : i - len + drafts);
        const RowStats* shares = static_cast<const RowStats*>(a.workspace) + row * parts.per_row;
        RowStats st = {Softmax::none(), -INFINITY, -1};
        for (int c = lane; c < parts.per_row; c += 32) {
            const RowStats u = shares[c];
            st.q.add(u.q, by);
            take(st.value, st.best, u.value, u.best);
        }
        st.q = warp_softmax(st.q, by);
        if (kGreedy)
            warp_best(st.value, st.best);
        if (lane == 0)
            whole[i] = st;
    }
    __syncthreads();

    // The first refused token.
    auto ok = [](const RowStats& s) { return s.q.sum > 0.0f && s.q.sum < INFINITY && s.q.max < INFINITY; };
    if (threadIdx.x < len) {
        const int i = threadIdx.x, token = a.tokens[b * drafts + i];
        bool accept = false;
        if (token >= 0 && token < vocab) {
            if (kGreedy) {
                accept = ok(whole[i]) && token == whole[i].best;
            } else {
                const RowStats &t = whole[i], &d = whole[point ? 0 : len + 1 + i];
                const float p = ex2((logit[0][i] - t.q.max) * scale) / t.q.sum;
                const float q = point ? 1.0f : ex2((logit[1][i] - d.q.max) * q_scale) / d.q.sum;
                accept = a.uniforms[b * drafts + i] * q < p;
            }
        }
        if (!accept)
            atomicMin(&refused, i);
    }
    __syncthreads();
    const int n = refused;
    const RowStats st = whole[n];
    int token = -1;
    if (ok(st)) {  // alike for all CTAs of the sequence
        if (kGreedy) {
            token = st.best;
        } else {
            const int without = n < len && point ? a.tokens[b * drafts + n] : -1;
            const bool minus = n < len && !point;
            const Packs<T> s(target_row(n), vocab);
            const T* q = minus ? draft_row(n) : nullptr;
            const float* noise = a.noise + b * a.ldn;
            const float inv = 1.0f / st.q.sum;
            const Softmax d = whole[minus ? len + 1 + n : 0].q;
            const float q_inv = 1.0f / d.sum;
            // Whether the rows' packs begin with the same elements, so that all come by whole 16-byte loads.
            const bool wide = ((reinterpret_cast<uint64_t>(noise - s.shift) | (minus ? reinterpret_cast<uint64_t>(q - s.shift) : 0)) & 15) == 0;
            float best = -1.0f;
            int at = -1;
            // r / e for r = max(p - q, 0) (kMinus) or p, as a product with the reciprocal (good to about 2^-22, and
            // the same for the same r and e). The products of p and q are rounded by themselves: fused with the
            // difference, equal distributions would leave a residue of rounding size in the place of 0.
            const uint64_t scale2 = pair(scale, scale), from2 = pair(-st.q.max, -st.q.max);
            const uint64_t q_scale2 = pair(q_scale, q_scale), q_from2 = pair(-d.max, -d.max);
            auto score2 = [&](auto subtract, uint64_t t, uint64_t u, float2 e) {
                const float2 x = halves(mul2(add2(t, from2), scale2));
                float2 r = make_float2(__fmul_rn(ex2(x.x), inv), __fmul_rn(ex2(x.y), inv));
                if constexpr (decltype(subtract)::value) {
                    const float2 y = halves(mul2(add2(u, q_from2), q_scale2));
                    r.x = __fsub_rn(r.x, __fmul_rn(ex2(y.x), q_inv));
                    r.y = __fsub_rn(r.y, __fmul_rn(ex2(y.y), q_inv));
                }
                return halves(mul2(pair(r.x, r.y), pair(rcp(e.x), rcp(e.y))));
            };
            // The race over packs start, start + stride, ... of the row; `skip` is a token that has no part in it.
            auto race = [&](auto subtract, auto whole_packs, int start, int stride, int skip, bool ends) {
                constexpr bool kMinus = decltype(subtract)::value, kWide = decltype(whole_packs)::value;
                for (int i = s.inside + start; i < s.end; i += stride) {
                    const int j = s.element(i);
                    const uint4 packed = s.load(i);
                    uint64_t t[kPairs<T>];
                    float u[N], e[N], sc[N], top = 0.0f;
                    if constexpr (kWide) {
                        if constexpr (kMinus)
                            load_beside(u, q, j);
                        load_beside(e, noise, j);
                    } else {
                        if constexpr (kMinus)
                            load_window(u, q, j, vocab);
                        load_window(e, noise, j, vocab);
                    }
                    unpack_pairs<T>(packed, t);
#pragma unroll
                    for (int k = 0; k < kPairs<T>; ++k) {
                        const float2 x = score2(subtract, t[k], kMinus ? pair(u[2 * k], u[2 * k + 1]) : 0, make_float2(e[2 * k], e[2 * k + 1]));
                        sc[2 * k] = x.x, sc[2 * k + 1] = x.y;
                    }
                    if (static_cast<unsigned>(skip - j) < N)
#pragma unroll
                        for (int k = 0; k < N; ++k)
                            sc[k] = j + k == skip ? 0.0f : sc[k];
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        top = fmaxf(top, sc[k]);
                    if (top > best && top > 0.0f) {  // of equals the lower token: later packs are higher
                        best = top;
#pragma unroll
                        for (int k = N - 1; k >= 0; --k)
                            at = sc[k] == top ? j + k : at;
                    }
                }
                // The ends' elements, a lane each.
                if (ends && warp == kWarps - 1 && lane < 2 * N) {
                    const int j = lane < N ? (s.inside ? lane - s.shift : -1) : s.element(s.end) + lane - N;
                    if (j >= 0 && j < vocab && j != skip) {
                        const float t = to_f32(s.row[j]), u = kMinus ? to_f32(q[j]) : 0.0f;
                        const float sc = score2(subtract, pair(t, t), pair(u, u), make_float2(noise[j], noise[j])).x;
                        if (sc > 0.0f)
                            take(best, at, sc, j);
                    }
                }
                // The CTA's best, to every thread.
                __syncwarp();
                warp_best(best, at);
                __syncthreads();  // a race before has read these
                if (lane == 0)
                    values[warp] = best, where[warp] = at;
                __syncthreads();
                best = values[lane % kWarps], at = where[lane % kWarps];
                warp_best(best, at);
            };
            using Yes = std::true_type;
            using No = std::false_type;
            const int start = rank * kThreads + threadIdx.x, stride = ctas * kThreads;
            if (minus && wide)
                race(Yes(), Yes(), start, stride, -1, rank == 0);
            else if (minus)
                race(Yes(), No(), start, stride, -1, rank == 0);
            else if (wide)
                race(No(), Yes(), start, stride, without, rank == 0);
            else
                race(No(), No(), start, stride, without, rank == 0);
            if (ctas > 1) {
                // The last CTA of the sequence to come here has all of them. (Which one that is changes nothing.)
                Races& races = races_of(a, parts)[b];
                if (threadIdx.x == 0) {
                    races.value[rank] = best, races.token[rank] = at;
                    __threadfence();
                    last = atomicAdd(&races.done, 1u) == static_cast<unsigned>(ctas) - 1;
                    __threadfence();
                }
                __syncthreads();
                if (!last)
                    return;
                best = -1.0f, at = -1;
                for (int c = lane; c < ctas; c += 32)
                    take(best, at, __ldcg(&races.value[c]), __ldcg(&races.token[c]));
                warp_best(best, at);
            }
            if (at < 0)  // p - q is nowhere positive: from p
                race(No(), No(), threadIdx.x, kThreads, -1, true);
            token = at;
        }
    }
    if (ctas > 1 && !ok(st) && rank)
        return;
    for (int i = threadIdx.x; i <= drafts; i += kThreads) {
        const int said = i < n ? a.tokens[b * drafts + i] : i == n ? token : -1;
        a.out[b * (drafts + 1) + i] = said;
        if (a.logprobs)
            a.logprobs[b * (drafts + 1) + i] =
                said < 0 ? 0.0f
                         : (((i < n ? logit[0][i] : to_f32(target_row(i)[said])) - whole[i].q.max) * scale -
                            log2f(whole[i].q.sum)) * kLn2;
    }
    if (threadIdx.x == 0)
        a.accepted[b] = n;
}

int check_sizes(int64_t batch, int64_t drafts, int64_t vocab)
{
    if (batch < 0 || drafts < 0 || vocab < 0)
        return fail_with(GEMM_ERR_ARG, "negative size");
    if (drafts > ROWOP_VERIFY_MAX_DRAFTS)
        return fail_with(GEMM_ERR_ARG, "drafts %lld is above %d", (long long)drafts, ROWOP_VERIFY_MAX_DRAFTS);
    if (batch > (1 << 20))
        return fail_with(GEMM_ERR_ARG, "batch %lld is above 2^20", (long long)batch);
    if (batch > 0 && (vocab < 1 || vocab > (INT64_C(1) << 30)))
        return fail_with(GEMM_ERR_ARG, "vocab %lld is not within 1 .. 2^30", (long long)vocab);
    return GEMM_OK;
}

int check(const rowop_verify_args* a)
{
    if (!a)
        return fail_with(GEMM_ERR_ARG, "args is NULL");
    const int rc = check_sizes(a->batch, a->drafts, a->vocab);
    if (rc || a->batch == 0)
        return rc;
    if (!type_ok(a->logits_type))
        return fail_with(GEMM_ERR_ARG, "bad type");
    if (!(a->temperature >= 0.0f) || a->temperature > 3e38f)
        return fail_with(GEMM_ERR_ARG, "temperature must be finite and not below 0");
    const bool greedy = a->temperature == 0.0f, draft = a->draft && !greedy;
    if (draft && (!(a->draft_temperature > 0.0f) || a->draft_temperature > 3e38f))
        return fail_with(GEMM_ERR_ARG, "draft_temperature must be finite and above 0");
    if (!a->target || !a->accepted || !a->out || (a->drafts > 0 && !a->tokens) ||
        (!greedy && (!a->noise || (a->drafts > 0 && !a->uniforms))))
        return fail_with(GEMM_ERR_ARG, "target, tokens, uniforms, noise, accepted or out is NULL");
    if (a->ldt < a->vocab || (draft && a->ldq < a->vocab) || (!greedy && a->ldn < a->vocab))
        return fail_with(GEMM_ERR_ARG, "row stride below vocab");
    if (!aligned(a->target, type_bytes(a->logits_type)) || !aligned(a->draft, type_bytes(a->logits_type)) ||
        !aligned(a->tokens, 4) || !aligned(a->lengths, 4) || !aligned(a->uniforms, 4) || !aligned(a->noise, 4) ||
        !aligned(a->accepted, 4) || !aligned(a->out, 4) || !aligned(a->logprobs, 4) || !aligned(a->workspace, 16))
        return fail_with(GEMM_ERR_ALIGN, "a pointer is not aligned to its elements, or workspace not to 16 bytes");
    if (!a->workspace || a->workspace_bytes < rowop_verify_workspace(a->batch, a->drafts, a->vocab))
        return fail_with(GEMM_ERR_ARG, "workspace is NULL or below rowop_verify_workspace()");
    return GEMM_OK;
}

template <typename T, bool kGreedy>
cudaError_t launch(const rowop_verify_args& a, cudaStream_t s)
{
    const bool draft = a.draft && !kGreedy;
    const Parts parts = parts_of(a.batch, a.drafts, a.vocab);
    const int64_t items = a.batch * (a.drafts + 1 + (draft ? a.drafts : 0)) * parts.per_row, ctas_wanted = (items + kWarps - 1) / kWarps;
    const unsigned grid = static_cast<unsigned>(ctas_wanted < kCtas ? ctas_wanted : kCtas);
    sat_verify_rows_kernel<T, kGreedy><<<grid, kThreads, 0, s>>>(a, parts);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    const int ctas = kGreedy ? 1 : racers_of(a.batch, a.vocab);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sat_verify_draw_kernel<T, kGreedy>, a, parts, ctas);
}

template <typename T>
cudaError_t launch_as(const rowop_verify_args& a, cudaStream_t s)
{
    return a.temperature == 0.0f ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

extern "C" {

int64_t rowop_verify_workspace(int64_t batch, int64_t drafts, int64_t vocab)
{
    set_last_error("");
    const int rc = check_sizes(batch, drafts, vocab);
    if (rc || batch == 0)
        return rc;
    return batch * ((2 * drafts + 1) * parts_of(batch, drafts, vocab).per_row * static_cast<int64_t>(sizeof(RowStats)) +
                    static_cast<int64_t>(sizeof(Races)));
}

int rowop_verify(const rowop_verify_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->batch == 0)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = args->logits_type == GEMM_C_F32    ? launch_as<float>(*args, s)
                          : args->logits_type == GEMM_C_BF16 ? launch_as<__nv_bfloat16>(*args, s)
                                                             : launch_as<__half>(*args, s);
    return e == cudaSuccess ? GEMM_OK
                            : fail_with(GEMM_ERR_LAUNCH, "launching the verification: %s", cudaGetErrorString(e));
}

}  // extern "C"
