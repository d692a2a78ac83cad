// Host-side interface between the C ABI (capi_step.cu) and the kernels around
// the linear log-probability in a training step.
#pragma once
#include "ll_internal.h"

namespace ll {

// --- embedding lookup and its gradient (embed_kernels.cu) ---------------------
struct EmbedArgs {
    const void* rows;       // lookup: the table; gradient: grad_out
    int64_t ld_rows;
    int dtype;              // of rows
    const int64_t* tokens;  // [N]
    int64_t N, D, V, v0;
    float scale;
    void* table;            // lookup: out; gradient: grad_weight
    int64_t ld_table;
    int table_dtype;
};
cudaError_t launch_embed_fwd(const EmbedArgs& a, cudaStream_t s);
size_t embed_bwd_bytes(int64_t N, int64_t D, int64_t V);
// The gradient's two parts, in this order: the tokens sorted into the workspace
// (and, without accumulate, rows of no token set to +0), then the sums.  Up to 1024
// tokens the first does nothing and the second matches them in one launch.
cudaError_t launch_embed_sort(const EmbedArgs& a, int accumulate, void* ws, const DevInfo& dev,
                              cudaStream_t s);
cudaError_t launch_embed_bwd(const EmbedArgs& a, int accumulate, void* ws, const DevInfo& dev,
                             cudaStream_t s);

// --- policy loss (policy_kernels.cu) -------------------------------------------
struct PolicyArgs {
    const float *logp, *old, *ref, *adv;  // ref may be null
    const uint8_t* mask;                  // or null
    const int64_t* offs;                  // [n_seqs + 1] or null
    int64_t n_seqs, N;
    float log_lo[2], log_hi[2];  // log(1 - clip_low), log(1 + clip_high): hi, lo parts
    float bound_lo, bound_hi;    // 1 - clip_low, 1 + clip_high
    double beta_d, denominator;
    float beta;
    float *stats, *grad;
};
constexpr int kPolicyBlocks = 304;  // most blocks, and so partial sums, of the loss kernel
struct PolicyWs {
    float2 part[3 * kPolicyBlocks];  // hi, lo
    int tokens[kPolicyBlocks];  // unmasked tokens of each block
    unsigned done, pad[3];      // blocks whose partial sums are written
    unsigned long long full;    // sequences that have an unmasked token
    unsigned long long pad2;    // the sequences' counts follow
};
size_t policy_ws_bytes(int64_t n_seqs);
cudaError_t launch_policy_loss(const PolicyArgs& a, void* workspace, cudaStream_t s);

// --- gradient norm and clipping (grad_kernels.cu) ------------------------------
constexpr int kMaxTensors = 512;      // tensors of one launch
constexpr int kGradMaxBlocks = 1024;  // most blocks, and so partial sums, of one launch
// norm[0] = the norm of the list.
cudaError_t launch_grad_norm(const ll_tensor* t, int64_t count, float* norm, void* ws,
                             int num_sms, cudaStream_t s);
// The list scaled by min(1, max_norm / (norm + 1e-6)): by norm[0], or with
// `compute` by the list's own, written to norm[0].
cudaError_t launch_grad_clip(const ll_tensor* t, int64_t count, float max_norm, bool compute,
                             float* norm, void* ws, int num_sms, cudaStream_t s);

}  // namespace ll
