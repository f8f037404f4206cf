// Verification of drafted tokens and the draw of the next one (include/rowops.h).
//
// A cluster of CTAs takes a sequence. Its CTAs go through their shares of the
// sequence's rows (each logit read once, 16 bytes a load, reduced to a
// maximum and a sum of exponentials), put the rows' softmaxes together
// through distributed shared memory, decide alike which token is the first
// refused, and race through their shares of that one row. HBM bandwidth
// bounds large batches; one sequence is a chain of latencies: the launch, a
// load, two exchanges and a second load.
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kMaxCluster = 16;
constexpr int kMaxRows = 2 * ROWOP_VERIFY_MAX_DRAFTS + 1;

// What is kept of a row (or of a CTA's or warp's share of it): its softmax,
// and for the greedy choice its largest value's lowest token.
struct __align__(16) RowStats {
    Softmax q;
    float value;
    int best;

    __device__ __forceinline__ void add(const RowStats& o, float scale);
};

// The larger value, or of equals the lower index; an index of -1 is none.
__device__ __forceinline__ void take(float& v, int& at, float v2, int at2)
{
    if (at2 >= 0 && (at < 0 || v2 > v || (v2 == v && at2 < at)))
        v = v2, at = at2;
}

__device__ __forceinline__ void RowStats::add(const RowStats& o, float scale)
{
    q.add(o.q, scale);
    take(value, best, o.value, o.best);
}

__device__ __forceinline__ void warp_best(float& v, int& at)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(v, at, __shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, at, o));
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint4& v)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
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

// Eight (or four) elements of another row of the same tokens, by one or two
// 16-byte loads where they lie on the boundaries for it.
template <int N, typename T>
__device__ __forceinline__ void load_beside(float (&v)[N], const T* row, int j, bool wide)
{
    if (wide) {
#pragma unroll
        for (int h = 0; h < N / kPer16<T>; ++h) {
            float u[kPer16<T>];
            unpack16<T>(*reinterpret_cast<const uint4*>(row + j + h * kPer16<T>), u);
#pragma unroll
            for (int e = 0; e < kPer16<T>; ++e)
                v[h * kPer16<T> + e] = u[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[e] = to_f32(row[j + e]);
    }
}

template <typename T, int NT, bool kGreedy>
__global__ void __launch_bounds__(NT, 1024 / NT) sat_verify_kernel(const __grid_constant__ rowop_verify_args a, int ctas)
{
    constexpr int N = kPer16<T>, kWarps = NT / 32;
    extern __shared__ RowStats stats[];  // [rows][kWarps], then [rows][ctas]
    __shared__ RowStats whole[kMaxRows];  // of the target's rows, then the draft's
    __shared__ float logit[2][ROWOP_VERIFY_MAX_DRAFTS];  // the target's and the draft's at the drafted tokens
    __shared__ RowStats races[kMaxCluster];
    __shared__ float values[kWarps];
    __shared__ int where[kWarps];
    __shared__ int refused;
    const int rank = blockIdx.x % ctas, drafts = static_cast<int>(a.drafts), vocab = static_cast<int>(a.vocab);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t b = blockIdx.x / ctas;
    const int len = a.lengths ? min(max(a.lengths[b], 0), drafts) : drafts;
    const bool point = kGreedy || !a.draft;
    // A greedy target's log probabilities are at temperature 1.
    const float scale = kGreedy ? kLog2e : kLog2e / a.temperature, q_scale = point ? 0.0f : kLog2e / a.draft_temperature;
    const int rows = len + 1 + (point ? 0 : len);
    RowStats* across = stats + rows * kWarps;
    auto target_row = [&](int i) { return static_cast<const T*>(a.target) + (b * (drafts + 1) + i) * a.ldt; };
    auto draft_row = [&](int i) { return static_cast<const T*>(a.draft) + (b * drafts + i) * a.ldq; };
    if (ctas > 1)
        cluster_arrive();  // waited for before the first store to another CTA, which has to have started by then
    if (threadIdx.x < len) {
        const int i = threadIdx.x, token = a.tokens[b * drafts + i];
        const bool there = token >= 0 && token < vocab;
        logit[0][i] = there ? to_f32(target_row(i)[token]) : -INFINITY;
        logit[1][i] = there && !point ? to_f32(draft_row(i)[token]) : 0.0f;
    }
    if (threadIdx.x == 0)
        refused = len;

    // The shares' softmaxes.
    for (int i = 0; i < rows; ++i) {
        const Packs<T> s(i <= len ? target_row(i) : draft_row(i - len - 1), vocab);
        const float by = i <= len ? scale : q_scale;
        RowStats st = {Softmax::none(), -INFINITY, -1};
        RunningSoftmax run;
        auto add = [&](const uint4& w, int pack) {
            if (kGreedy && largest<T>(w) > st.value) {
                float v[N];
                unpack16<T>(w, v);
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (v[e] > st.value)
                        st.value = v[e], st.best = s.element(pack) + e;
            }
            run.add<T>(w, by);
        };
        constexpr int U = 4;
        int j = s.inside + rank * NT + threadIdx.x;
        for (; j + (U - 1) * ctas * NT < s.end; j += U * ctas * NT) {
            uint4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = s.load(j + u * ctas * NT);
#pragma unroll
            for (int u = 0; u < U; ++u)
                add(w[u], j + u * ctas * NT);
        }
        for (; j < s.end; j += ctas * NT)
            add(s.load(j), j);
        st.q = run.whole();
        // The ends' elements, a lane each.
        if (rank == 0 && warp == kWarps - 1 && lane < 2 * N) {
            const int c = lane < N ? (s.inside ? lane - s.shift : -1) : s.element(s.end) + lane - N;
            if (c >= 0 && c < vocab) {
                const float v = to_f32(s.row[c]);
                if (kGreedy && v > -INFINITY)
                    take(st.value, st.best, v, c);
                st.q.add(v, by);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            RowStats u;
            u.q.max = __shfl_down_sync(0xffffffffu, st.q.max, o);
            u.q.sum = __shfl_down_sync(0xffffffffu, st.q.sum, o);
            if (kGreedy) {
                u.value = __shfl_down_sync(0xffffffffu, st.value, o);
                u.best = __shfl_down_sync(0xffffffffu, st.best, o);
                st.add(u, by);
            } else {
                st.q.add(u.q, by);
            }
        }
        if (lane == 0)
            stats[i * kWarps + warp] = st;
    }
    __syncthreads();
    // Put together: the CTA's warps, then the cluster's CTAs, in order.
    auto scale_of = [&](int i) { return i <= len ? scale : q_scale; };
    if (ctas > 1) {
        __syncwarp();
        cluster_wait();
    }
    for (int i = threadIdx.x; i < rows; i += NT) {
        RowStats st = stats[i * kWarps];
        for (int w = 1; w < kWarps; ++w)
            st.add(stats[i * kWarps + w], scale_of(i));
        if (ctas == 1)
            whole[i] = st;
        else
            for (int c = 0; c < ctas; ++c)
                st_cluster_v4(map_to_cta(smem_u32(&across[i * ctas + rank]), c), *reinterpret_cast<const uint4*>(&st));
    }
    if (ctas > 1) {
        __syncwarp();
        cluster_sync();
        for (int i = threadIdx.x; i < rows; i += NT) {
            RowStats st = across[i * ctas];
            for (int c = 1; c < ctas; ++c)
                st.add(across[i * ctas + c], scale_of(i));
            whole[i] = st;
        }
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
    if (ok(st)) {  // alike for all CTAs of the cluster
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
            const bool q_wide = minus && (reinterpret_cast<uint64_t>(q - s.shift) & 15) == 0;
            const bool noise_wide = (reinterpret_cast<uint64_t>(noise - s.shift) & 15) == 0;
            // The race of max(p - q, 0), and where that is nowhere positive, of p.
            for (int pass = 0; pass < 2 && token < 0; ++pass) {
                float best = -1.0f;
                int at = -1;
                auto run = [&](float t, float u, float e, int j) {
                    // Products rounded by themselves: fused with the difference, equal distributions
                    // would leave a residue of rounding size in the place of 0.
                    const float p = __fmul_rn(ex2((t - st.q.max) * scale), inv);
                    float r = p;
                    if (pass == 0)
                        r = minus ? p - __fmul_rn(ex2((u - d.max) * q_scale), q_inv) : j == without ? 0.0f : p;
                    // The quotient only where it may be the largest.
                    if (r > 0.0f && r >= best * e * 0.999999f)
                        take(best, at, r / e, j);
                };
                for (int i = s.inside + rank * NT + threadIdx.x; i < s.end; i += ctas * NT) {
                    float t[N], u[N] = {}, e[N];
                    const int j = s.element(i);
                    unpack16<T>(s.load(i), t);
                    if (minus)
                        load_beside(u, q, j, q_wide);
                    load_beside(e, noise, j, noise_wide);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        run(t[k], u[k], e[k], j + k);
                }
                if (rank == 0 && warp == kWarps - 1 && lane < 2 * N) {
                    const int j = lane < N ? (s.inside ? lane - s.shift : -1) : s.element(s.end) + lane - N;
                    if (j >= 0 && j < vocab)
                        run(to_f32(s.row[j]), minus ? to_f32(q[j]) : 0.0f, noise[j], j);
                }
                warp_best(best, at);
                __syncthreads();  // the pass before has read these
                if (lane == 0)
                    values[warp] = best, where[warp] = at;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w)
                    take(best, at, values[w], where[w]);
                if (ctas > 1) {
                    if (threadIdx.x < ctas) {
                        const uint4 v = make_uint4(__float_as_uint(best), static_cast<uint32_t>(at), 0, 0);
                        st_cluster_v4(map_to_cta(smem_u32(&races[rank]), threadIdx.x), v);
                    }
                    __syncwarp();
                    cluster_sync();
                    for (int c = 0; c < ctas; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(&races[c]);
                        take(best, at, __uint_as_float(v.x), static_cast<int>(v.y));
                    }
                    if (pass == 0 && at < 0) {  // `races` is read before it is written again
                        __syncwarp();
                        cluster_sync();
                    }
                }
                token = at;
            }
        }
    }
    if (rank)
        return;
    for (int i = threadIdx.x; i <= drafts; i += NT) {
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

template <typename T, int NT, bool kGreedy>
cudaError_t launch_one(const rowop_verify_args& a, int ctas, cudaStream_t s)
{
    const bool draft = a.draft && !kGreedy;
    const int rows = static_cast<int>(a.drafts + 1 + (draft ? a.drafts : 0));
    auto kernel = sat_verify_kernel<T, NT, kGreedy>;
    static Prepared prepared;
    const cudaError_t e = prepared.once(reinterpret_cast<const void*>(kernel),
                                        kMaxRows * (NT / 32 + kMaxCluster) * static_cast<int>(sizeof(RowStats)));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.batch * ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = rows * (NT / 32 + ctas) * sizeof(RowStats);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, ctas);
}

template <typename T>
cudaError_t launch(const rowop_verify_args& a, cudaStream_t s)
{
    // Four CTAs of 256 threads an SM, 608 in all, where the batch gives them;
    // where even clusters of 16 leave SMs idle, the CTAs have 1024 threads.
    int ctas = 1;
    while (ctas < kMaxCluster && a.batch * ctas * 2 <= 608 && a.vocab * static_cast<int64_t>(sizeof(T)) > ctas * 4096)
        ctas *= 2;
    const bool few = a.batch * ctas <= 152;
    if (a.temperature == 0.0f)
        return few ? launch_one<T, 1024, true>(a, ctas, s) : launch_one<T, 256, true>(a, ctas, s);
    return few ? launch_one<T, 1024, false>(a, ctas, s) : launch_one<T, 256, false>(a, ctas, s);
}

}  // namespace

extern "C" {

int64_t rowop_verify_workspace(int64_t batch, int64_t drafts, int64_t vocab)
{
    set_last_error("");
    const int rc = check_sizes(batch, drafts, vocab);
    return rc ? rc : batch * (2 * drafts + 1) * static_cast<int64_t>(sizeof(RowStats));
}

int rowop_verify(const rowop_verify_args* args, void* stream)
{
    set_last_error("");
    const int rc = check(args);
    if (rc || args->batch == 0)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = args->logits_type == GEMM_C_F32    ? launch<float>(*args, s)
                          : args->logits_type == GEMM_C_BF16 ? launch<__nv_bfloat16>(*args, s)
                                                             : launch<__half>(*args, s);
    return e == cudaSuccess ? GEMM_OK
                            : fail_with(GEMM_ERR_LAUNCH, "launching the verification: %s", cudaGetErrorString(e));
}

}  // extern "C"
