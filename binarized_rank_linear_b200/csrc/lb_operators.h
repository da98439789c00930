// lb_operators.h - host-side interfaces between the C ABI of the operators beside
// the projection (lb_api_operators.cu) and their kernels.  Not installed; not part
// of the ABI.
#pragma once

#include "lb_internal.h"

namespace lb {

// ---------------------------------------------------------------- adapters (lb_adapters.cu)
// Low-rank adapters of many requests (lb_adapters_forward, _backward),
// already validated.
constexpr int kMaxAdapters = LB_MAX_ADAPTERS;
constexpr int kAdapterSmallTokens = LB_ADAPTERS_SMALL_TOKENS;
struct AdapterProj {
    const uint16_t *a, *b;
    const float *scale;
    const int32_t *ranks;
    int rank, n_out;
    const uint16_t *base;  // never null: y itself for an update in place
    int64_t ldbase;
    uint16_t *y;
    int64_t ldy;
};
struct AdaptersArgs {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *ids;
    int tokens, n_in, count, nproj;
    AdapterProj proj[kMaxSiblings];
    void *workspace;
};
struct AdaptersBwdArgs {
    const uint16_t *x, *dy;
    int64_t ldx, lddy;
    const int32_t *ids;
    int tokens, n_in, n_out, count, rank;
    const uint16_t *a, *b;
    const float *scale;
    const int32_t *ranks;
    const uint16_t *dx_base;  // dx itself for an update in place
    int64_t lddxbase;
    uint16_t *dx;  // may be null
    int64_t lddx;
    float *da, *db;
    void *workspace;
};
size_t adapters_workspace_bytes(int tokens, int n_in, int count, int nproj, const int *ranks);
cudaError_t adapters_forward(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream);
size_t adapters_backward_workspace_bytes(int tokens, int count, int rank);
cudaError_t adapters_backward(const AdaptersBwdArgs &a, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t adapters_prepare_device(const DeviceInfo &dev);
// Past the small batches (from 177 tokens on, where the pool has one adapter;
// always past kAdapterSmallTokens), and the backward pass (lb_adapters_mma.cu).
size_t adapters_mma_workspace_bytes(int tokens, int count, int nproj, const int *ranks);
cudaError_t adapters_mma_forward(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream);
size_t adapters_mma_backward_workspace_bytes(int tokens, int count, int rank);
cudaError_t adapters_mma_backward(const AdaptersBwdArgs &a, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t adapters_mma_prepare_device(const DeviceInfo &dev);

// ---------------------------------------------------------------- heads (lb_heads.cu)
// Per-head norm and position rotation (lb_heads_norm_rotate and its backward
// pass), already validated.  Forward: in -> out.  Backward: in, dout -> out
// (the gradient of in) and dweight.
constexpr int kMaxHeadGroups = LB_MAX_SIBLINGS;
constexpr int kMaxHeads = 4096;     // of a call's tensors together
constexpr int kMaxHeadCtas = 1024;  // most rows of dweight partials
struct HeadGroup {
    const uint16_t *in, *dout, *weight;
    int64_t ld_in, ld_dout, ld_out;
    uint16_t *out;
    float *dweight;
    int heads;
};
struct HeadsArgs {
    HeadGroup group[kMaxHeadGroups];
    int ngroups, tokens, head_dim, rotary_dim, pairs;
    const int32_t *positions;
    const float *inv_freq;
    float eps;
};
size_t heads_backward_workspace_bytes(int head_dim);
cudaError_t heads_forward(const HeadsArgs &a, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t heads_backward(const HeadsArgs &a, float *workspace, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t heads_prepare_device(const DeviceInfo &dev);

}  // namespace lb
