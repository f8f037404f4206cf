// Verification of drafted tokens and the draw of the next one (include/rowops.h).
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 512, kWarps = kThreads / 32;

// What the first kernel leaves of a row: its softmax, and its first largest token.
struct RowStats {
    float max, sum;
    int best;
    int unused;
};

// The larger value, or of equals the lower index.
__device__ __forceinline__ void take(float& v, int& at, float v2, int at2)
{
    if (at2 >= 0 && (at < 0 || v2 > v || (v2 == v && at2 < at)))
        v = v2, at = at2;
}

// The largest value over a CTA and the lowest index that has it (-1 for none), to every thread.
__device__ __forceinline__ void cta_best(float& v, int& at, float* values, int* where)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(v, at, __shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, at, o));
    if ((threadIdx.x & 31) == 0)
        values[threadIdx.x >> 5] = v, where[threadIdx.x >> 5] = at;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < kWarps ? values[lane] : 0.0f;
    at = lane < kWarps ? where[lane] : -1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        take(v, at, __shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, at, o));
}

__device__ __forceinline__ int length_of(const rowop_verify_args& a, int64_t b)
{
    const int drafts = static_cast<int>(a.drafts);
    return a.lengths ? min(max(a.lengths[b], 0), drafts) : drafts;
}

// Scales of the exponents: a greedy target's log probabilities are at temperature 1.
__device__ __forceinline__ float target_scale(const rowop_verify_args& a)
{
    return a.temperature > 0.0f ? kLog2e / a.temperature : kLog2e;
}

// One CTA a row: the target's rows (all sequences'), then the draft's.
template <typename T>
__global__ void __launch_bounds__(kThreads) sat_verify_rows_kernel(const __grid_constant__ rowop_verify_args a)
{
    __shared__ Softmax scratch[kWarps];
    __shared__ float values[kWarps];
    __shared__ int where[kWarps];
    const int64_t rows = a.batch * (a.drafts + 1), row = blockIdx.x;
    const bool target = row < rows;
    const int64_t b = target ? row / (a.drafts + 1) : (row - rows) / a.drafts;
    const int i = static_cast<int>(target ? row % (a.drafts + 1) : (row - rows) % a.drafts), len = length_of(a, b);
    if (target ? i > len : i >= len)
        return;
    const T* s = target ? static_cast<const T*>(a.target) + row * a.ldt : static_cast<const T*>(a.draft) + (row - rows) * a.ldq;
    const float scale = target ? target_scale(a) : kLog2e / a.draft_temperature;
    Softmax q;
    float v = 0.0f;
    int best = -1;
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const float x = to_f32(s[j]);
        take(v, best, x, j);
        q.add(x, scale);
    }
    q = cta_softmax<kThreads>(q, scale, scratch);
    cta_best(v, best, values, where);
    if (threadIdx.x == 0)
        static_cast<RowStats*>(a.workspace)[row] = {q.max, q.sum, best, 0};
}

// One CTA a sequence: the decisions, then the draw.
template <typename T>
__global__ void __launch_bounds__(kThreads) sat_verify_draw_kernel(const __grid_constant__ rowop_verify_args a)
{
    __shared__ float values[2][kWarps];
    __shared__ int where[2][kWarps];
    __shared__ int refused;
    const int64_t b = blockIdx.x, drafts = a.drafts;
    const RowStats* stats = static_cast<const RowStats*>(a.workspace);
    const RowStats* ts = stats + b * (drafts + 1);
    const RowStats* qs = stats + a.batch * (drafts + 1) + b * drafts;
    const float scale = target_scale(a), q_scale = kLog2e / a.draft_temperature;
    const int len = length_of(a, b);
    const bool greedy = a.temperature == 0.0f, point = greedy || !a.draft;
    auto target_row = [&](int i) { return static_cast<const T*>(a.target) + (b * (drafts + 1) + i) * a.ldt; };
    auto draft_row = [&](int i) { return static_cast<const T*>(a.draft) + (b * drafts + i) * a.ldq; };
    // Whether a row has a distribution: neither all -inf nor a NaN or +inf in it.
    auto ok = [](const RowStats& s) { return s.sum > 0.0f && s.sum < INFINITY && s.max < INFINITY; };
    if (threadIdx.x == 0)
        refused = len;
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += kThreads) {
        const int token = a.tokens[b * drafts + i];
        bool accept = false;
        if (token >= 0 && token < a.vocab) {
            if (greedy) {
                accept = ok(ts[i]) && token == ts[i].best;
            } else {
                const float p = exp2f((to_f32(target_row(i)[token]) - ts[i].max) * scale) / ts[i].sum;
                const float q = point ? 1.0f : exp2f((to_f32(draft_row(i)[token]) - qs[i].max) * q_scale) / qs[i].sum;
                accept = a.uniforms[b * drafts + i] * q < p;
            }
        }
        if (!accept)
            atomicMin(&refused, i);
    }
    __syncthreads();
    const int n = refused;
    const RowStats st = ts[n];
    const T* t = target_row(n);
    int token = -1;
    if (ok(st)) {
        if (greedy) {
            token = st.best;
        } else {
            // The race of max(p - q, 0), and that of p for where p - q is nowhere positive.
            const int without = n < len && point ? a.tokens[b * drafts + n] : -1;
            const bool minus = n < len && !point;
            const T* q = minus ? draft_row(n) : nullptr;
            const float inv = 1.0f / st.sum, q_max = minus ? qs[n].max : 0.0f, q_inv = minus ? 1.0f / qs[n].sum : 0.0f;
            const float* noise = a.noise + b * a.ldn;
            float v = 0.0f, all = 0.0f;
            int all_at = -1;
            for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
                // Products rounded by themselves: fused with the difference, equal distributions would leave a
                // residue of rounding size in the place of 0.
                const float p = __fmul_rn(exp2f((to_f32(t[j]) - st.max) * scale), inv);
                const float r = minus ? p - __fmul_rn(exp2f((to_f32(q[j]) - q_max) * q_scale), q_inv)
                                      : j == without ? 0.0f : p;
                if (r > 0.0f)
                    take(v, token, r / noise[j], j);
                if (p > 0.0f)
                    take(all, all_at, p / noise[j], j);
            }
            cta_best(v, token, values[0], where[0]);
            cta_best(all, all_at, values[1], where[1]);
            if (token < 0)
                token = all_at;
        }
    }
    for (int i = threadIdx.x; i <= drafts; i += kThreads) {
        const int said = i < n ? a.tokens[b * drafts + i] : i == n ? token : -1;
        a.out[b * (drafts + 1) + i] = said;
        if (a.logprobs)
            a.logprobs[b * (drafts + 1) + i] =
                said < 0 ? 0.0f
                         : (to_f32(target_row(i)[said]) - ts[i].max) * (scale / kLog2e) - logf(ts[i].sum);
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

template <typename T>
cudaError_t launch(const rowop_verify_args& a, cudaStream_t s)
{
    const bool draft = a.draft && a.temperature > 0.0f;
    const int64_t rows = a.batch * (a.drafts + 1) + (draft ? a.batch * a.drafts : 0);
    sat_verify_rows_kernel<T><<<static_cast<unsigned>(rows), kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    sat_verify_draw_kernel<T><<<static_cast<unsigned>(a.batch), kThreads, 0, s>>>(a);
    return cudaGetLastError();
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
