// lb_api_operators.cu - the C ABI (include/lb.h) of the operators beside the
// projection: adapters of many requests, per-head norm and rotation.  Argument
// checks and dispatch; apart from lb_api.cu, so that figures of the projection's
// own calls do not depend on it.
#include <cstdint>

#include <cuda_runtime.h>

#include "lb.h"
#include "lb_operators.h"

namespace {

using lb::aligned16;
using lb::aligned4;
using lb::device_info;
using lb::kMaxDim;
using lb::kMaxTokens;
constexpr int64_t kMaxAdapterTokens = int64_t(1) << 20, kMaxAdapterLd = int64_t(1) << 30;

}  // namespace

cudaError_t lb::operators_prepare_device(const DeviceInfo &dev)
{
    const cudaError_t e = adapters_prepare_device(dev);
    return e != cudaSuccess ? e : heads_prepare_device(dev);
}

// The sizes of a pool; `sizes_only` leaves its pointers unchecked.
static lb_status check_pool(const lb_adapters *p, bool sizes_only)
{
    if (!p || p->count < 1 || p->rank < 1) return LB_ERR_INVALID_ARGUMENT;
    if (p->count > LB_MAX_ADAPTERS || p->rank % 8 != 0 || p->rank > LB_MAX_ADAPTER_RANK) return LB_ERR_UNSUPPORTED_SHAPE;
    if (sizes_only) return LB_OK;
    if (!p->a || !p->b) return LB_ERR_INVALID_ARGUMENT;
    if (!aligned16(p->a) || !aligned16(p->b) || !aligned4(p->scale) || !aligned4(p->ranks)) return LB_ERR_MISALIGNED;
    return LB_OK;
}

// Everything an adapters call checks on the host except the workspace; fills `a`.
static lb_status build_adapters(const uint16_t *x, int64_t tokens, int64_t n_in, int64_t ldx, const int32_t *ids,
                                int nproj, const lb_adapter_projection *proj, bool sizes_only, lb::AdaptersArgs *a)
{
    if (tokens < 0 || n_in <= 0 || nproj < 1 || nproj > LB_MAX_SIBLINGS || !proj) return LB_ERR_INVALID_ARGUMENT;
    if (n_in % 32 != 0 || n_in > kMaxDim || tokens > kMaxAdapterTokens) return LB_ERR_UNSUPPORTED_SHAPE;
    if (!sizes_only) {
        if (!x || !ids || ldx < n_in) return LB_ERR_INVALID_ARGUMENT;
        if (ldx > kMaxAdapterLd) return LB_ERR_UNSUPPORTED_SHAPE;
        if (ldx % 8 != 0 || !aligned16(x) || !aligned4(ids)) return LB_ERR_MISALIGNED;
    }
    *a = lb::AdaptersArgs{};
    a->x = x;
    a->ldx = ldx;
    a->ids = ids;
    a->tokens = (int)tokens;
    a->n_in = (int)n_in;
    a->nproj = nproj;
    for (int j = 0; j < nproj; ++j) {
        const lb_adapter_projection &pj = proj[j];
        lb::AdapterProj &d = a->proj[j];
        const lb_status st = check_pool(pj.adapters, sizes_only);
        if (st != LB_OK) return st;
        if (pj.n_out <= 0 || pj.adapters->count != proj[0].adapters->count) return LB_ERR_INVALID_ARGUMENT;
        if (pj.n_out % 32 != 0 || pj.n_out > kMaxDim) return LB_ERR_UNSUPPORTED_SHAPE;
        d.rank = (int)pj.adapters->rank;
        d.n_out = (int)pj.n_out;
        if (sizes_only) continue;
        if (!pj.y || pj.ldy < pj.n_out || (pj.base && pj.ldbase < pj.n_out)) return LB_ERR_INVALID_ARGUMENT;
        if (pj.base == pj.y && pj.ldbase != pj.ldy) return LB_ERR_INVALID_ARGUMENT;
        if (pj.ldy > kMaxAdapterLd || (pj.base && pj.ldbase > kMaxAdapterLd)) return LB_ERR_UNSUPPORTED_SHAPE;
        if (pj.ldy % 8 != 0 || !aligned16(pj.y) || (pj.base && (pj.ldbase % 8 != 0 || !aligned16(pj.base))))
            return LB_ERR_MISALIGNED;
        d.a = pj.adapters->a;
        d.b = pj.adapters->b;
        d.scale = pj.adapters->scale;
        d.ranks = pj.adapters->ranks;
        d.base = pj.base ? pj.base : pj.y;
        d.ldbase = pj.base ? pj.ldbase : pj.ldy;
        d.y = pj.y;
        d.ldy = pj.ldy;
    }
    a->count = (int)proj[0].adapters->count;
    return LB_OK;
}

static size_t adapters_need(const lb::AdaptersArgs &a)
{
    int ranks[LB_MAX_SIBLINGS];
    for (int j = 0; j < a.nproj; ++j) ranks[j] = a.proj[j].rank;
    return lb::adapters_workspace_bytes(a.tokens, a.n_in, a.count, a.nproj, ranks);
}

size_t lb_adapters_workspace_bytes(int64_t tokens, int64_t n_in, int nproj, const lb_adapter_projection *proj)
{
    lb::AdaptersArgs a;
    if (build_adapters(nullptr, tokens, n_in, n_in, nullptr, nproj, proj, true, &a) != LB_OK || tokens == 0) return 0;
    return adapters_need(a);
}

lb_status lb_adapters_forward(const uint16_t *x, int64_t tokens, int64_t n_in, int64_t ldx, const int32_t *ids,
                              int nproj, const lb_adapter_projection *proj, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    if (tokens < 0 || n_in <= 0 || nproj < 1 || nproj > LB_MAX_SIBLINGS || !proj) return LB_ERR_INVALID_ARGUMENT;
    if (tokens == 0) return LB_OK;
    lb::AdaptersArgs a;
    lb_status st = build_adapters(x, tokens, n_in, ldx, ids, nproj, proj, false, &a);
    if (st != LB_OK) return st;
    const size_t need = adapters_need(a);
    if (need > 0 && !workspace) return LB_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return LB_ERR_WORKSPACE_TOO_SMALL;
    if (workspace && !aligned16(workspace)) return LB_ERR_MISALIGNED;
    a.workspace = workspace;
    lb::DeviceInfo dev;
    st = device_info(&dev);
    if (st != LB_OK) return st;
    if (lb::adapters_forward(a, dev, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return LB_ERR_CUDA;
    }
    return LB_OK;
}

static bool adapters_backward_sizes(int64_t tokens, int64_t n_in, int64_t n_out)
{
    return n_in % 32 == 0 && n_out % 32 == 0 && n_in <= kMaxDim && n_out <= kMaxDim && tokens <= kMaxAdapterTokens;
}

size_t lb_adapters_backward_workspace_bytes(int64_t tokens, int64_t n_in, int64_t n_out, int64_t count, int64_t rank)
{
    const lb_adapters pool = {nullptr, nullptr, nullptr, nullptr, count, rank};
    if (tokens <= 0 || n_in <= 0 || n_out <= 0 || !adapters_backward_sizes(tokens, n_in, n_out) ||
        check_pool(&pool, true) != LB_OK)
        return 0;
    return lb::adapters_backward_workspace_bytes((int)tokens, (int)count, (int)rank);
}

lb_status lb_adapters_backward(const uint16_t *x, const uint16_t *dy, int64_t tokens, int64_t n_in, int64_t n_out,
                               int64_t ldx, int64_t lddy, const int32_t *ids, const lb_adapters *adapters,
                               const uint16_t *dx_base, int64_t lddxbase, uint16_t *dx, int64_t lddx, float *da,
                               float *db, void *workspace, size_t workspace_bytes, void *stream)
{
    if (tokens < 0 || n_in <= 0 || n_out <= 0 || !da || !db) return LB_ERR_INVALID_ARGUMENT;
    if (tokens > 0 && (!x || !dy || !ids)) return LB_ERR_INVALID_ARGUMENT;
    if (ldx < n_in || lddy < n_out || (dx && lddx < n_in) || (dx && dx_base && lddxbase < n_in))
        return LB_ERR_INVALID_ARGUMENT;
    if (dx && dx_base == dx && lddxbase != lddx) return LB_ERR_INVALID_ARGUMENT;
    if (!adapters_backward_sizes(tokens, n_in, n_out)) return LB_ERR_UNSUPPORTED_SHAPE;
    if (ldx > kMaxAdapterLd || lddy > kMaxAdapterLd || (dx && (lddx > kMaxAdapterLd || (dx_base && lddxbase > kMaxAdapterLd))))
        return LB_ERR_UNSUPPORTED_SHAPE;
    lb_status st = check_pool(adapters, false);
    if (st != LB_OK) return st;
    if (ldx % 8 != 0 || lddy % 8 != 0 || !aligned16(x) || !aligned16(dy) || !aligned4(ids)) return LB_ERR_MISALIGNED;
    if (dx && (lddx % 8 != 0 || !aligned16(dx))) return LB_ERR_MISALIGNED;
    if (dx && dx_base && (lddxbase % 8 != 0 || !aligned16(dx_base))) return LB_ERR_MISALIGNED;
    if (!aligned16(da) || !aligned16(db)) return LB_ERR_MISALIGNED;
    lb::AdaptersBwdArgs b{};
    b.count = (int)adapters->count;
    b.rank = (int)adapters->rank;
    const size_t need = tokens > 0 ? lb::adapters_backward_workspace_bytes((int)tokens, b.count, b.rank)
                                   : 0;
    if (need > 0 && !workspace) return LB_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return LB_ERR_WORKSPACE_TOO_SMALL;
    if (workspace && !aligned16(workspace)) return LB_ERR_MISALIGNED;
    lb::DeviceInfo dev;
    st = device_info(&dev);
    if (st != LB_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        const size_t per = sizeof(float) * (size_t)b.count * (size_t)b.rank;
        if (cudaMemsetAsync(da, 0, per * (size_t)n_in, s) != cudaSuccess ||
            cudaMemsetAsync(db, 0, per * (size_t)n_out, s) != cudaSuccess) {
            cudaGetLastError();
            return LB_ERR_CUDA;
        }
        return LB_OK;
    }
    b.x = x;
    b.dy = dy;
    b.ldx = ldx;
    b.lddy = lddy;
    b.ids = ids;
    b.tokens = (int)tokens;
    b.n_in = (int)n_in;
    b.n_out = (int)n_out;
    b.a = adapters->a;
    b.b = adapters->b;
    b.scale = adapters->scale;
    b.ranks = adapters->ranks;
    b.dx_base = dx_base ? dx_base : dx;
    b.lddxbase = dx_base ? lddxbase : lddx;
    b.dx = dx;
    b.lddx = lddx;
    b.da = da;
    b.db = db;
    b.workspace = workspace;
    if (lb::adapters_backward(b, dev, s) != cudaSuccess) {
        cudaGetLastError();
        return LB_ERR_CUDA;
    }
    return LB_OK;
}

// What both heads calls check of their sizes, positions and frequencies (tokens > 0).
static lb_status check_heads(int64_t tokens, int64_t head_dim, int64_t rotary_dim, lb_rotation rotation,
                             const int32_t *positions, const float *inv_freq, float eps, lb::HeadsArgs *a)
{
    if (rotation != LB_ROTATE_HALVES && rotation != LB_ROTATE_PAIRS) return LB_ERR_INVALID_ARGUMENT;
    if (rotary_dim < 0 || rotary_dim > head_dim || !(eps >= 0.0f) || !(eps <= 3.0e38f)) return LB_ERR_INVALID_ARGUMENT;
    if (rotary_dim > 0 && tokens > 0 && (!positions || !inv_freq)) return LB_ERR_INVALID_ARGUMENT;
    if (head_dim % 8 != 0 || head_dim > 256 || rotary_dim % 8 != 0 || tokens > kMaxTokens) return LB_ERR_UNSUPPORTED_SHAPE;
    if (!aligned4(positions) || !aligned4(inv_freq)) return LB_ERR_MISALIGNED;
    a->tokens = (int)tokens;
    a->head_dim = (int)head_dim;
    a->rotary_dim = (int)rotary_dim;
    a->pairs = rotation == LB_ROTATE_PAIRS;
    a->positions = positions;
    a->inv_freq = inv_freq;
    a->eps = eps;
    return LB_OK;
}

constexpr int64_t kMaxHeadsLd = int64_t(1) << 30;

lb_status lb_heads_norm_rotate(int64_t tokens, int64_t head_dim, int64_t rotary_dim, lb_rotation rotation,
                               const int32_t *positions, const float *inv_freq, float eps, int ntensors,
                               const lb_heads *tensors, void *stream)
{
    if (tokens < 0 || head_dim <= 0 || ntensors < 1 || ntensors > LB_MAX_SIBLINGS || !tensors)
        return LB_ERR_INVALID_ARGUMENT;
    lb::HeadsArgs a{};
    lb_status st = check_heads(tokens, head_dim, rotary_dim, rotation, positions, inv_freq, eps, &a);
    if (st != LB_OK) return st;
    if (tokens == 0) return LB_OK;
    a.ngroups = ntensors;
    int64_t total = 0;
    for (int g = 0; g < ntensors; ++g) {
        const lb_heads &t = tensors[g];
        if (t.heads < 1 || !t.in || !t.out) return LB_ERR_INVALID_ARGUMENT;
        total += t.heads;
        if (t.heads > lb::kMaxHeads || total > lb::kMaxHeads) return LB_ERR_UNSUPPORTED_SHAPE;
        if (t.ld_in > kMaxHeadsLd || t.ld_out > kMaxHeadsLd) return LB_ERR_UNSUPPORTED_SHAPE;
        if (t.ld_in < t.heads * head_dim || t.ld_out < t.heads * head_dim) return LB_ERR_INVALID_ARGUMENT;
        if (t.in == t.out && t.ld_in != t.ld_out) return LB_ERR_INVALID_ARGUMENT;
        if (t.ld_in % 8 != 0 || t.ld_out % 8 != 0 || !aligned16(t.in) || !aligned16(t.out) || !aligned16(t.weight))
            return LB_ERR_MISALIGNED;
        lb::HeadGroup &d = a.group[g];
        d.in = t.in;
        d.ld_in = t.ld_in;
        d.weight = t.weight;
        d.out = t.out;
        d.ld_out = t.ld_out;
        d.heads = (int)t.heads;
    }
    lb::DeviceInfo dev;
    st = device_info(&dev);
    if (st != LB_OK) return st;
    if (lb::heads_forward(a, dev, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return LB_ERR_CUDA;
    }
    return LB_OK;
}

size_t lb_heads_backward_workspace_bytes(int64_t head_dim)
{
    if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 256) return 0;
    return lb::heads_backward_workspace_bytes((int)head_dim);
}

lb_status lb_heads_norm_rotate_backward(int64_t tokens, int64_t head_dim, int64_t rotary_dim, lb_rotation rotation,
                                        const int32_t *positions, const float *inv_freq, float eps, int ntensors,
                                        const lb_heads_grad *tensors, void *workspace, size_t workspace_bytes,
                                        void *stream)
{
    if (tokens < 0 || head_dim <= 0 || ntensors < 1 || ntensors > LB_MAX_SIBLINGS || !tensors)
        return LB_ERR_INVALID_ARGUMENT;
    lb::HeadsArgs a{};
    lb_status st = check_heads(tokens, head_dim, rotary_dim, rotation, positions, inv_freq, eps, &a);
    if (st != LB_OK) return st;
    a.ngroups = ntensors;
    int64_t total = 0;
    bool sums = false;
    for (int g = 0; g < ntensors; ++g) {
        const lb_heads_grad &t = tensors[g];
        // `in` is read for the norm alone
        if (t.heads < 1 || (t.dweight && !t.weight)) return LB_ERR_INVALID_ARGUMENT;
        total += t.heads;
        if (t.heads > lb::kMaxHeads || total > lb::kMaxHeads) return LB_ERR_UNSUPPORTED_SHAPE;
        sums = sums || t.dweight != nullptr;
        lb::HeadGroup &d = a.group[g];
        d.heads = (int)t.heads;
        d.dweight = t.dweight;
        if (!aligned16(t.weight) || !aligned4(t.dweight)) return LB_ERR_MISALIGNED;
        if (tokens == 0) continue;
        const int64_t row = t.heads * head_dim;
        if (t.ld_in > kMaxHeadsLd || t.ld_dout > kMaxHeadsLd || t.ld_din > kMaxHeadsLd) return LB_ERR_UNSUPPORTED_SHAPE;
        if (!t.dout || !t.din || t.ld_dout < row || t.ld_din < row) return LB_ERR_INVALID_ARGUMENT;
        if (t.weight && (!t.in || t.ld_in < row)) return LB_ERR_INVALID_ARGUMENT;
        if (t.din == t.dout && t.ld_din != t.ld_dout) return LB_ERR_INVALID_ARGUMENT;
        if (t.weight && t.din == t.in && t.ld_din != t.ld_in) return LB_ERR_INVALID_ARGUMENT;
        if (t.ld_dout % 8 != 0 || t.ld_din % 8 != 0 || !aligned16(t.dout) || !aligned16(t.din)) return LB_ERR_MISALIGNED;
        if (t.weight && (t.ld_in % 8 != 0 || !aligned16(t.in))) return LB_ERR_MISALIGNED;
        d.in = t.in;
        d.ld_in = t.ld_in;
        d.weight = t.weight;
        d.dout = t.dout;
        d.ld_dout = t.ld_dout;
        d.out = t.din;
        d.ld_out = t.ld_din;
    }
    if (tokens > 0 && sums) {
        if (!workspace) return LB_ERR_INVALID_ARGUMENT;
        if (workspace_bytes < lb::heads_backward_workspace_bytes((int)head_dim)) return LB_ERR_WORKSPACE_TOO_SMALL;
        if (!aligned16(workspace)) return LB_ERR_MISALIGNED;
    }
    lb::DeviceInfo dev;
    st = device_info(&dev);
    if (st != LB_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (tokens == 0) {
        for (int g = 0; g < ntensors; ++g)
            if (tensors[g].dweight &&
                cudaMemsetAsync(tensors[g].dweight, 0, sizeof(float) * (size_t)head_dim, s) != cudaSuccess) {
                cudaGetLastError();
                return LB_ERR_CUDA;
            }
        return LB_OK;
    }
    if (lb::heads_backward(a, static_cast<float *>(workspace), dev, s) != cudaSuccess) {
        cudaGetLastError();
        return LB_ERR_CUDA;
    }
    return LB_OK;
}
