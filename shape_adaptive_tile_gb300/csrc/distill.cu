// Distillation from a teacher's top logits and its gradient (include/rowops.h).
#include "rows.cuh"

namespace {

using namespace sat;
using namespace sat::rows;

constexpr int kThreads = 512;

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

// One CTA a row: the teacher's entries into shared memory, the student's
// softmax in one pass over its logits, the gradient in a second.
template <typename T, bool kForward>
__global__ void __launch_bounds__(kThreads) sat_distill_kernel(const __grid_constant__ rowop_distill_args a)
{
    __shared__ Softmax scratch[kThreads / 32];
    __shared__ float sums[2 * 2 * (kThreads / 32)];
    __shared__ int id[ROWOP_DISTILL_MAX_K];    // -1 for an absent entry
    __shared__ float p[ROWOP_DISTILL_MAX_K];   // the teacher's probability
    __shared__ float at[ROWOP_DISTILL_MAX_K];  // the student's logit
    int turn = 0;
    const int k = static_cast<int>(a.k);
    const float scale = kLog2e / a.temperature, inv_t = 1.0f / a.temperature;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        __syncthreads();  // the previous row's entries are no longer read
        const T* s = static_cast<const T*>(a.logits) + r * a.ldl;
        T* d = a.dlogits ? static_cast<T*>(a.dlogits) + r * a.ldd : nullptr;
        const float weight = a.weight ? a.weight[r] : 1.0f;
        Softmax t;
        for (int i = threadIdx.x; i < k; i += kThreads) {
            const int token = a.ids[r * a.ldi + i];
            const float v = teacher_logit(a, r * a.ldt + i);
            const bool there = token >= 0 && token < a.vocab && v != -INFINITY;
            id[i] = there ? token : -1;
            p[i] = v;
            if (there)
                t.add(v, scale);
        }
        t = cta_softmax<kThreads>(t, scale, scratch);
        if (weight == 0.0f || t.max == -INFINITY) {
            if (kForward && threadIdx.x == 0) {
                a.loss[r] = 0.0f;
                if (a.lse)
                    a.lse[r] = 0.0f;
            }
            if (d)
                for (int j = threadIdx.x; j < a.vocab; j += kThreads)
                    d[j] = from_f32<T>(0.0f);
            continue;
        }
        Softmax q;
        if (kForward) {
            for (int j = threadIdx.x; j < a.vocab; j += kThreads)
                q.add(to_f32(s[j]), scale);
            __syncthreads();  // scratch has been read
            q = cta_softmax<kThreads>(q, scale, scratch);
        } else {
            q.max = a.lse[r] * a.temperature;
            q.sum = 1.0f;
        }
        // log p_i = (T_i - L') / t with L' the largest of T, and so on.
        const float top = a.teacher_lse ? a.teacher_lse[r] : t.max * inv_t + logf(t.sum);
        const float log_sum = logf(q.sum);
        float sum[2] = {0.0f, 0.0f};  // of p, and of p (log p - log q)
        for (int i = threadIdx.x; i < k; i += kThreads) {
            float pi = 0.0f;
            if (id[i] >= 0) {
                const float log_p = a.teacher_lse ? fmaf(p[i], inv_t, -top) : (p[i] - t.max) * inv_t - logf(t.sum);
                pi = expf(log_p);
                at[i] = to_f32(s[id[i]]);
                if (pi > 0.0f)
                    sum[1] += pi * (log_p - ((at[i] - q.max) * inv_t - log_sum));
                sum[0] += pi;
            }
            p[i] = pi;
        }
        row_sums<kThreads>(sum, sums, turn);
        if (kForward && threadIdx.x == 0) {
            a.loss[r] = weight * a.temperature * a.temperature * sum[1];
            if (a.lse)
                a.lse[r] = q.max * inv_t + log_sum;
        }
        if (!d)
            continue;
        const float c = (a.dloss ? a.dloss[r] : 1.0f) * weight * a.temperature;
        const float log2_sum = log_sum * kLog2e;
        auto whole = [&](float v) { return sum[0] * exp2f(fmaf(v - q.max, scale, -log2_sum)); };
        for (int j = threadIdx.x; j < a.vocab; j += kThreads)
            d[j] = from_f32<T>(c * whole(to_f32(s[j])));
        __syncthreads();
        // The teacher's tokens, each once: by the first of the entries that name it.
        for (int i = threadIdx.x; i < k; i += kThreads) {
            if (id[i] < 0)
                continue;
            bool first = true;
            float pi = 0.0f;
            for (int l = 0; l < k; ++l)
                if (id[l] == id[i]) {
                    first = first && l >= i;
                    pi += p[l];
                }
            if (first)
                d[id[i]] = from_f32<T>(c * (whole(at[i]) - pi));
        }
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

template <bool kForward>
int run(const rowop_distill_args* a, void* stream)
{
    set_last_error("");
    const int rc = check(a, kForward);
    if (rc || a->rows == 0)
        return rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>(a->rows < (1 << 20) ? a->rows : (1 << 20));
    if (a->logits_type == GEMM_C_F32)
        sat_distill_kernel<float, kForward><<<grid, kThreads, 0, s>>>(*a);
    else if (a->logits_type == GEMM_C_BF16)
        sat_distill_kernel<__nv_bfloat16, kForward><<<grid, kThreads, 0, s>>>(*a);
    else
        sat_distill_kernel<__half, kForward><<<grid, kThreads, 0, s>>>(*a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? GEMM_OK
                            : fail_with(GEMM_ERR_LAUNCH, "launching the distillation kernel: %s", cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int rowop_distill(const rowop_distill_args* args, void* stream) { return run<true>(args, stream); }

int rowop_distill_backward(const rowop_distill_args* args, void* stream) { return run<false>(args, stream); }

}  // extern "C"
