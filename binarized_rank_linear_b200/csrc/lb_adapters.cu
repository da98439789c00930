// lb_adapters.cu - low-rank adapters of many requests beside a shared
// projection: the dispatch by token count and the CUDA-core kernels for small
// batches.
//
//     y[m] = base[m] + s_i B_i (A_i x[m]),  i = ids[m]
//
// At decode a batch reads the adapters its tokens use and little else: 2 r (n_in
// + n_out) bytes an adapter against 4 r (n_in + n_out) operations a token, far
// below what DRAM or the launches cost, so the products run on CUDA cores in
// fp32 straight from the weights as they lie.  Two launches:
//   shrink  a CTA takes up to kGroup tokens of one adapter and a slice of n_in;
//           a warp per row of A, 16 bytes a lane, the slice's x of those tokens
//           in shared memory; v partials [slice][token][rank] in fp32
//   expand  a CTA takes the same tokens and 256 outputs: a thread per output
//           row of B, the tokens' v (the slices added in order, scaled) in
//           shared memory
// Tokens that share an adapter thus read its weights once per kGroup of them,
// wherever they stand in the batch.  Both launches fetch their weights before
// they wait for the launch they depend on (programmatic dependent launch).
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_internal.h"

namespace lb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 8;       // tokens of one adapter that a CTA takes together
constexpr int kStep = 256;      // columns of A a warp reads at once (16 bytes a lane)
constexpr int kMaxSteps = 4;    // steps of a shrink CTA's slice
static_assert(kAdapterSmallTokens <= kThreads, "one thread for each token looks for its adapter");

struct SmallParams {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *ids;
    int tokens, n_in, count, steps, slices;
    AdapterProj proj[kMaxSiblings];
    float *part[kMaxSiblings];        // [slice][token][rank]
    int chunk0[kMaxSiblings + 1];     // expand: first 256-output chunk of each projection
    int nproj;
    int *status;
};

// The tokens of this CTA: blockIdx.y = m leads a group when the number of
// earlier tokens with m's adapter is a multiple of kGroup; it then takes m and
// the next ones, up to kGroup.  Returns their number, 0 for a CTA that leads
// none; `id` is the adapter, or -1.  One thread per token; ends in a barrier.
struct Group {
    int tok[kGroup];
};
__device__ __forceinline__ int find_group(const SmallParams &p, Group &g, uint32_t *masks, int &id)
{
    const int m = blockIdx.y, t = threadIdx.x, lane = t & 31, w = t >> 5;
    int mine = __ldg(p.ids + m);
    if (mine >= p.count) {
        if (t == 0 && blockIdx.x == 0 && blockIdx.z == 0) set_status(p.status, LB_ERR_INVALID_ARGUMENT);
        mine = -1;
    }
    id = mine < 0 ? -1 : mine;
    int other = -2;
    if (t < p.tokens) {
        other = __ldg(p.ids + t);
        if (other < 0 || other >= p.count) other = -1;
    }
    const bool eq = other == id;
    const uint32_t mask = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) masks[w] = mask;
    __syncthreads();
    int before = 0, total = 0, upto = 0;  // matches before m, in all, and before t
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const uint32_t k = masks[i];
        total += __popc(k);
        before += __popc(i < (m >> 5) ? k : i == (m >> 5) ? k & ((1u << (m & 31)) - 1u) : 0u);
        upto += __popc(i < w ? k : i == w ? k & ((1u << lane) - 1u) : 0u);
    }
    if (before % kGroup != 0) return 0;
    const int n = min(kGroup, total - before);
    if (eq && upto >= before && upto < before + n) g.tok[upto - before] = t;
    __syncthreads();
    return n;
}

__device__ __forceinline__ int rank_of(const AdapterProj &P, int id)
{
    return P.ranks == nullptr ? P.rank : max(0, min(P.rank, __ldg(P.ranks + id)));
}

__device__ __forceinline__ void fma8(float &acc, const uint4 &w, const uint4 &x)
{
    const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc += __uint_as_float(a[i] << 16) * __uint_as_float(b[i] << 16);
        acc += __uint_as_float(a[i] & 0xffff0000u) * __uint_as_float(b[i] & 0xffff0000u);
    }
}

// grid (slices, tokens, projections)
__global__ void __launch_bounds__(kThreads) small_shrink_kernel(const __grid_constant__ SmallParams p)
{
    __shared__ Group grp;
    __shared__ uint32_t masks[kWarps];
    __shared__ uint4 xs[kGroup][kMaxSteps * 32];
    int id;
    const int n = find_group(p, grp, masks, id);
    const AdapterProj &P = p.proj[blockIdx.z];
    const int rank = n > 0 && id >= 0 ? rank_of(P, id) : 0;
    if (rank == 0) {  // uniform over the CTA
        pdl_wait();
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k0 = blockIdx.x * p.steps * kStep + 8 * lane;
    const uint16_t *a = P.a + (int64_t)id * P.rank * p.n_in;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load_row = [&](int r, uint4(&w)[kMaxSteps]) {
#pragma unroll
        for (int s = 0; s < kMaxSteps; ++s) {
            const int k = k0 + s * kStep;
            w[s] = r < rank && s < p.steps && k < p.n_in ? ldg_early_v4(a + (int64_t)r * p.n_in + k) : zero;
        }
    };
    uint4 w0[kMaxSteps], w1[kMaxSteps];
    load_row(warp, w0);  // weights do not depend on the launch before
    load_row(warp + kWarps, w1);
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < n * p.steps * 32; i += kThreads) {
        const int g = i / (p.steps * 32), c = i - g * (p.steps * 32);
        const int k = blockIdx.x * p.steps * kStep + 8 * c;
        xs[g][c] = k < p.n_in ? *reinterpret_cast<const uint4 *>(p.x + (int64_t)grp.tok[g] * p.ldx + k) : zero;
    }
    __syncthreads();
    float *part = p.part[blockIdx.z] + (int64_t)blockIdx.x * p.tokens * P.rank;
    for (int r = warp; r < rank; r += 2 * kWarps) {
        if (r != warp) {
            load_row(r, w0);
            load_row(r + kWarps, w1);
        }
        for (int g = 0; g < n; ++g) {
            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
            for (int s = 0; s < kMaxSteps; ++s) {
                if (s < p.steps) {
                    const uint4 xv = xs[g][32 * s + lane];
                    fma8(s0, w0[s], xv);
                    fma8(s1, w1[s], xv);
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            }
            if (lane == 0) {
                float *v = part + (int64_t)grp.tok[g] * P.rank + r;
                v[0] = s0;
                if (r + kWarps < rank) v[kWarps] = s1;
            }
        }
    }
}

// grid (256-output chunks of every projection, tokens)
__global__ void __launch_bounds__(kThreads) small_expand_kernel(const __grid_constant__ SmallParams p)
{
    __shared__ Group grp;
    __shared__ uint32_t masks[kWarps];
    __shared__ alignas(16) float vs[kGroup][LB_MAX_ADAPTER_RANK];
    int id;
    const int n = find_group(p, grp, masks, id);
    int j = 0;
    while (j + 1 < p.nproj && (int)blockIdx.x >= p.chunk0[j + 1]) ++j;
    const AdapterProj &P = p.proj[j];
    const int o = ((int)blockIdx.x - p.chunk0[j]) * kThreads + threadIdx.x;
    const int rank = n > 0 && id >= 0 ? rank_of(P, id) : 0;
    if (n == 0 || (rank == 0 && P.base == P.y)) {  // uniform over the CTA
        pdl_wait();
        return;
    }
    const bool on = o < P.n_out;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const uint16_t *b = P.b + ((int64_t)max(id, 0) * P.n_out + o) * P.rank;
    constexpr int kPre = 4;
    uint4 w[kPre];
#pragma unroll
    for (int q = 0; q < kPre; ++q) w[q] = on && 8 * q < rank ? ldg_early_v4(b + 8 * q) : zero;
    const float scale = P.scale != nullptr && rank > 0 ? __ldg(P.scale + id) : 1.0f;
    pdl_wait();
    pdl_launch_dependents();
    float acc[kGroup];
    if (rank > 0) {
        const int r8 = (rank + 7) & ~7;
        for (int i = threadIdx.x; i < n * r8; i += kThreads) {
            const int g = i / r8, r = i - g * r8;
            const float *v = p.part[j] + (int64_t)grp.tok[g] * P.rank + r;
            float s = 0.0f;
            if (r < rank)
                for (int q = 0; q < p.slices; ++q) s += v[(int64_t)q * p.tokens * P.rank];
            vs[g][r] = s * scale;
        }
        __syncthreads();
#pragma unroll
        for (int g = 0; g < kGroup; ++g) acc[g] = 0.0f;
        for (int q0 = 0; 8 * q0 < rank; q0 += kPre) {
            if (q0 > 0) {
#pragma unroll
                for (int q = 0; q < kPre; ++q) w[q] = on && 8 * (q0 + q) < rank ? ldg_early_v4(b + 8 * (q0 + q)) : zero;
            }
#pragma unroll
            for (int q = 0; q < kPre; ++q) {
                if (8 * (q0 + q) < rank) {
                    const uint32_t k[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[2 * i] = __uint_as_float(k[i] << 16);
                        f[2 * i + 1] = __uint_as_float(k[i] & 0xffff0000u);
                    }
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) {
                        if (g < n) {
                            const float4 v0 = *reinterpret_cast<const float4 *>(&vs[g][8 * (q0 + q)]);
                            const float4 v1 = *reinterpret_cast<const float4 *>(&vs[g][8 * (q0 + q) + 4]);
                            acc[g] += f[0] * v0.x + f[1] * v0.y + f[2] * v0.z + f[3] * v0.w + f[4] * v1.x + f[5] * v1.y +
                                      f[6] * v1.z + f[7] * v1.w;
                        }
                    }
                }
            }
        }
    }
    if (!on) return;
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
        if (g < n) {
            const int64_t t = grp.tok[g];
            const uint16_t y = P.base[t * P.ldbase + o];
            P.y[t * P.ldy + o] = rank > 0 ? float_to_bf16_bits(bf16_bits_to_float(y) + acc[g]) : y;
        }
    }
}

// Columns of n_in per shrink CTA, in steps of 256: as many as leave about two
// CTAs for every SM.
int small_steps(int tokens, int n_in, int nproj)
{
    const int all = (n_in + kStep - 1) / kStep;
    int steps = kMaxSteps;
    while (steps > 1 && tokens * nproj * ((all + steps - 1) / steps) < 296) --steps;
    return steps;
}
int small_slices(int tokens, int n_in, int nproj)
{
    const int cols = small_steps(tokens, n_in, nproj) * kStep;
    return (n_in + cols - 1) / cols;
}

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, const SmallParams &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t small_adapters(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    const int M = a.tokens;
    SmallParams p{};
    p.x = a.x;
    p.ldx = a.ldx;
    p.ids = a.ids;
    p.tokens = M;
    p.n_in = a.n_in;
    p.count = a.count;
    p.nproj = a.nproj;
    p.steps = small_steps(M, a.n_in, a.nproj);
    p.slices = small_slices(M, a.n_in, a.nproj);
    p.status = dev.status;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    for (int j = 0; j < a.nproj; ++j) {
        p.proj[j] = a.proj[j];
        p.part[j] = reinterpret_cast<float *>(ws);
        ws += align256(sizeof(float) * (size_t)p.slices * (size_t)M * (size_t)a.proj[j].rank);
        p.chunk0[j + 1] = p.chunk0[j] + (a.proj[j].n_out + kThreads - 1) / kThreads;
    }
    cudaError_t e = launch_pdl(small_shrink_kernel, dim3((unsigned)p.slices, (unsigned)M, (unsigned)a.nproj), p, stream);
    if (e != cudaSuccess) return e;
    return launch_pdl(small_expand_kernel, dim3((unsigned)p.chunk0[a.nproj], (unsigned)M), p, stream);
}

size_t small_workspace(int M, int n_in, int nproj, const int *ranks)
{
    size_t b = 0;
    for (int j = 0; j < nproj; ++j)
        b += align256(sizeof(float) * (size_t)small_slices(M, n_in, nproj) * (size_t)M * (size_t)ranks[j]);
    return b;
}

}  // namespace

size_t adapters_workspace_bytes(int tokens, int n_in, int count, int nproj, const int *ranks)
{
    return tokens > kAdapterSmallTokens ? adapters_mma_workspace_bytes(tokens, count, nproj, ranks)
                                        : small_workspace(tokens, n_in, nproj, ranks);
}

cudaError_t adapters_prepare_device(const DeviceInfo &dev) { return adapters_mma_prepare_device(dev); }

cudaError_t adapters_forward(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    return a.tokens > kAdapterSmallTokens ? adapters_mma_forward(a, dev, stream) : small_adapters(a, dev, stream);
}

size_t adapters_backward_workspace_bytes(int tokens, int count, int rank)
{
    return adapters_mma_backward_workspace_bytes(tokens, count, rank);
}

cudaError_t adapters_backward(const AdaptersBwdArgs &b, const DeviceInfo &dev, cudaStream_t stream)
{
    return adapters_mma_backward(b, dev, stream);
}

}  // namespace lb
