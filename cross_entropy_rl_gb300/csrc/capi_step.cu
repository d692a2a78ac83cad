// C ABI of the calls around the linear log-probability in a training step:
// argument validation and the launches of each call.  Declarations and the
// contract of every entry point: ll_linear_logp.h.
#include <math.h>

#include <algorithm>
#include <new>

#include "capi_common.h"
#include "step_internal.h"

namespace ll {
namespace {
// Bytes from the first to past the last element of [rows, cols] with row stride ld.
size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t es) {
    return (size_t(rows - 1) * size_t(ld) + size_t(cols)) * es;
}
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const char* x = static_cast<const char*>(a);
    const char* y = static_cast<const char*>(b);
    return x < y + nb && y < x + na;
}
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Validation shared by the embedding's two entry points; `table` has V rows,
// `batch` N rows.
int embed_checks(int64_t N, int64_t D, int64_t V, int64_t v0, int64_t ld_table, int64_t ld_batch,
                 float scale) {
    int st = check_sizes(N, D, V);
    if (st) return st;
    if (v0 < 0 || v0 > kMaxV - V || ld_table < D || ld_batch < D) return LL_ERR_SHAPE;
    if (ld_table > (int64_t(1) << 31) || ld_batch > (int64_t(1) << 31)) return LL_ERR_SHAPE;
    if (!(fabsf(scale) < INFINITY)) return LL_ERR_INVALID_ARG;
    return LL_OK;
}

// Validation of a tensor list; with `apart`, also that no two tensors overlap.
int check_tensors(const ll_tensor* t, int64_t count, bool apart, const void** any) {
    *any = nullptr;
    if (count < 0) return LL_ERR_SHAPE;
    if (count > 0 && !t) return LL_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        if (!dtype_ok(t[i].dtype)) return LL_ERR_DTYPE;
        if (t[i].n < 0 || t[i].n > (int64_t(1) << 48)) return LL_ERR_SHAPE;
        if (t[i].reserved != 0) return LL_ERR_INVALID_ARG;
        if (t[i].n == 0) continue;
        if (!t[i].data) return LL_ERR_INVALID_ARG;
        if (!aligned_to(t[i].data, esize(t[i].dtype))) return LL_ERR_ALIGN;
        *any = t[i].data;
    }
    if (!apart || count < 2) return LL_OK;
    uintptr_t end = 0;
    bool ascending = true;  // as views of one buffer mostly are
    for (int64_t i = 0; i < count && ascending; ++i) {
        if (t[i].n == 0) continue;
        const uintptr_t p = reinterpret_cast<uintptr_t>(t[i].data);
        ascending = p >= end;
        end = p + size_t(t[i].n) * esize(t[i].dtype);
    }
    if (ascending) return LL_OK;
    const ll_tensor** at = new (std::nothrow) const ll_tensor*[count];
    if (!at) return LL_ERR_INVALID_ARG;
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i)
        if (t[i].n > 0) at[n++] = t + i;
    std::sort(at, at + n, [](const ll_tensor* a, const ll_tensor* b) {
        return reinterpret_cast<uintptr_t>(a->data) < reinterpret_cast<uintptr_t>(b->data);
    });
    int st = LL_OK;
    for (int64_t i = 1; i < n; ++i)
        if (overlap(at[i - 1]->data, size_t(at[i - 1]->n) * esize(at[i - 1]->dtype), at[i]->data, 1))
            st = LL_ERR_INVALID_ARG;
    delete[] at;
    return st;
}
}  // namespace
}  // namespace ll

using namespace ll;

extern "C" {

int ll_embed_forward(const void* weight, int64_t ldw, int dtype, const int64_t* tokens, int64_t N,
                     int64_t D, int64_t V, int64_t v0, float scale, void* out, int64_t ld_out,
                     int out_dtype, void* stream) {
    if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return LL_ERR_DTYPE;
    if (!(out_dtype == dtype || out_dtype == LL_F32 || dtype == LL_F32)) return LL_ERR_DTYPE;
    int st = embed_checks(N, D, V, v0, ldw, ld_out, scale);
    if (st || N == 0) return st;
    if (!weight || !tokens || !out) return LL_ERR_INVALID_ARG;
    if (!aligned_to(weight, esize(dtype)) || !aligned_to(out, esize(out_dtype)) ||
        !aligned_to(tokens, 8))
        return LL_ERR_ALIGN;
    if (overlap(weight, span_bytes(V, D, ldw, esize(dtype)), out,
                span_bytes(N, D, ld_out, esize(out_dtype))))
        return LL_ERR_INVALID_ARG;
    DeviceGuard guard(weight);
    if (guard.err) return guard.err;
    DevInfo dev;
    if ((st = device_info(guard.dev, &dev))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Phase ph("embed_fwd", s);
    return cuda_status(launch_embed_fwd(
        EmbedArgs{weight, ldw, dtype, tokens, N, D, V, v0, scale, out, ld_out, out_dtype}, s));
}

size_t ll_embed_workspace_size(int64_t N, int64_t D, int64_t V) {
    if (N <= 0 || check_sizes(N, D, V)) return 0;
    return align_up(embed_bwd_bytes(N, D, V));
}

int ll_embed_backward(const void* grad_out, int64_t ldg, int dtype, const int64_t* tokens,
                      int64_t N, int64_t D, int64_t V, int64_t v0, float scale, int accumulate,
                      void* grad_weight, int64_t ldw, int dw_dtype, void* workspace,
                      size_t ws_bytes, void* stream) {
    if (!dtype_ok(dtype) || !(dw_dtype == dtype || dw_dtype == LL_F32)) return LL_ERR_DTYPE;
    int st = embed_checks(N, D, V, v0, ldw, ldg, scale);
    if (st) return st;
    if (accumulate & ~1) return LL_ERR_INVALID_ARG;
    if (!grad_weight) return LL_ERR_INVALID_ARG;
    if (!aligned_to(grad_weight, esize(dw_dtype))) return LL_ERR_ALIGN;
    if (N == 0 && accumulate) return LL_OK;
    if (N > 0) {
        if (!grad_out || !tokens) return LL_ERR_INVALID_ARG;
        if (!aligned_to(grad_out, esize(dtype)) || !aligned_to(tokens, 8)) return LL_ERR_ALIGN;
        if (overlap(grad_out, span_bytes(N, D, ldg, esize(dtype)), grad_weight,
                    span_bytes(V, D, ldw, esize(dw_dtype))))
            return LL_ERR_INVALID_ARG;
        if (!workspace || ws_bytes < ll_embed_workspace_size(N, D, V)) return LL_ERR_WORKSPACE;
        if (!aligned_to(workspace, kAlign)) return LL_ERR_WORKSPACE;
    }
    DeviceGuard guard(grad_weight);
    if (guard.err) return guard.err;
    DevInfo dev;
    if ((st = device_info(guard.dev, &dev))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0)
        return cuda_status(cudaMemset2DAsync(grad_weight, size_t(ldw) * esize(dw_dtype), 0,
                                             size_t(D) * esize(dw_dtype), size_t(V), s));
    const EmbedArgs a{grad_out, ldg, dtype, tokens, N, D, V, v0, scale, grad_weight, ldw, dw_dtype};
    {
        Phase ph("embed_sort", s);
        const cudaError_t e = launch_embed_sort(a, accumulate, workspace, dev, s);
        if (e != cudaSuccess) return cuda_status(e);
    }
    Phase ph("embed_grad", s);
    return cuda_status(launch_embed_bwd(a, accumulate, workspace, dev, s));
}

size_t ll_policy_workspace_size(int64_t N, int64_t n_seqs) {
    if (N <= 0 || n_seqs < 0) return 0;
    return align_up(policy_ws_bytes(n_seqs));
}

int ll_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                   const float* advantages, const uint8_t* mask, const int64_t* seq_offsets,
                   int64_t n_seqs, int64_t N, const ll_policy_options* opt, float* stats,
                   float* grad_logp, void* workspace, size_t ws_bytes, void* stream) {
    const ll_policy_options o = opt ? *opt : ll_policy_options{0.2, 0.2, 0.0, 0.0, {0, 0, 0, 0}};
    for (int r : o.reserved)
        if (r != 0) return LL_ERR_INVALID_ARG;
    if (!(o.clip_low >= 0 && o.clip_low < 1) || !(o.clip_high >= 0 && o.clip_high < INFINITY) ||
        !(o.kl_coef >= 0 && o.kl_coef < INFINITY) ||
        !(o.denominator >= 0 && o.denominator < INFINITY))
        return LL_ERR_INVALID_ARG;
    if (o.kl_coef > 0 && !ref_logp && N > 0) return LL_ERR_INVALID_ARG;
    if (N < 0 || N > (int64_t(1) << 31) - 256) return LL_ERR_SHAPE;
    if (n_seqs < 0 || n_seqs > (int64_t(1) << 31) - 256) return LL_ERR_SHAPE;
    if ((n_seqs > 0) != (seq_offsets != nullptr) || !stats) return LL_ERR_INVALID_ARG;
    if (!aligned_to(stats, 4)) return LL_ERR_ALIGN;
    if (N > 0) {
        if (!logp || !old_logp || !advantages || !grad_logp) return LL_ERR_INVALID_ARG;
        if (!aligned_to(logp, 4) || !aligned_to(old_logp, 4) || !aligned_to(ref_logp, 4) ||
            !aligned_to(advantages, 4) || !aligned_to(grad_logp, 4) || !aligned_to(seq_offsets, 8))
            return LL_ERR_ALIGN;
        if (!workspace || ws_bytes < ll_policy_workspace_size(N, n_seqs)) return LL_ERR_WORKSPACE;
        if (!aligned_to(workspace, kAlign)) return LL_ERR_WORKSPACE;
    }
    DeviceGuard guard(stats);
    if (guard.err) return guard.err;
    DevInfo dev;
    int st = device_info(guard.dev, &dev);
    if (st) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (N == 0) return cuda_status(cudaMemsetAsync(stats, 0, 16, s));
    Phase ph("policy_loss", s);
    const double lo = log1p(-o.clip_low), hi = log1p(o.clip_high);
    return cuda_status(launch_policy_loss(
        PolicyArgs{logp, old_logp, ref_logp, advantages, mask, seq_offsets, n_seqs, N,
                   {float(lo), float(lo - float(lo))}, {float(hi), float(hi - float(hi))},
                   float(1.0 - o.clip_low), float(1.0 + o.clip_high), o.kl_coef, o.denominator,
                   float(o.kl_coef), stats, grad_logp},
        workspace, s));
}

size_t ll_grad_norm_workspace_size(int64_t count) {
    if (count < 0) return 0;
    return align_up(size_t(cdiv(count, kMaxTensors) + 1) * kGradMaxBlocks * sizeof(double));
}

int ll_grad_norm(const ll_tensor* tensors, int64_t count, float* norm, void* workspace,
                 size_t ws_bytes, void* stream) {
    const void* any;
    int st = check_tensors(tensors, count, false, &any);
    if (st) return st;
    if (!norm) return LL_ERR_INVALID_ARG;
    if (!aligned_to(norm, 4)) return LL_ERR_ALIGN;
    if (!workspace || ws_bytes < ll_grad_norm_workspace_size(count)) return LL_ERR_WORKSPACE;
    if (!aligned_to(workspace, kAlign)) return LL_ERR_WORKSPACE;
    DeviceGuard guard(norm);
    if (guard.err) return guard.err;
    DevInfo dev;
    if ((st = device_info(guard.dev, &dev))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Phase ph("grad_norm", s);
    return cuda_status(launch_grad_norm(tensors, count, norm, workspace, dev.num_sms, s));
}

int ll_clip_grads(const ll_tensor* tensors, int64_t count, float max_norm, int norm_given,
                  float* norm, void* workspace, size_t ws_bytes, void* stream) {
    const void* any;
    int st = check_tensors(tensors, count, true, &any);
    if (st) return st;
    if (!(max_norm > 0.f) || (norm_given & ~1) || !norm) return LL_ERR_INVALID_ARG;
    if (!aligned_to(norm, 4)) return LL_ERR_ALIGN;
    if (!norm_given) {
        if (!workspace || ws_bytes < ll_grad_norm_workspace_size(count)) return LL_ERR_WORKSPACE;
        if (!aligned_to(workspace, kAlign)) return LL_ERR_WORKSPACE;
    }
    if (!any && norm_given) return LL_OK;
    DeviceGuard guard(norm);
    if (guard.err) return guard.err;
    DevInfo dev;
    if ((st = device_info(guard.dev, &dev))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Phase ph("grad_clip", s);
    return cuda_status(launch_grad_clip(tensors, count, max_norm, !norm_given, norm, workspace,
                                        dev.num_sms, s));
}

}  // extern "C"
