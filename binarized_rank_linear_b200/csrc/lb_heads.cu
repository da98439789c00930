// lb_heads.cu - per-head norm and position rotation of projected queries and
// keys, forward and backward.
//
// For one head x [d] of a token at position p, with norm weights w and the
// rotation's frequencies f [rd / 2]:
//     n = w (.) x / sqrt(mean(x^2) + eps)        (n = x without weights)
//     (out_a, out_b) = (n_a cos t - n_b sin t, n_b cos t + n_a sin t),  t = p f_k,
// over the pairs (a, b) = (k, k + rd/2) or (2k, 2k + 1); elements from rd on
// pass.  Backward, with dn the transposed rotation of dout and x^ = x rstd:
//     dw = sum dn (.) x^,   dx = rstd (w (.) dn - x^ mean(w (.) dn (.) x^)).
//
// Every element is read and written once and costs a few operations, so DRAM
// bounds both passes: 4 bytes an element forward, 6 backward.  The kernels
// therefore keep a head in one pass: L = 8, 16 or 32 lanes hold 8 elements
// each (both ends of a rotated pair in the same lane, so the rotation needs no
// exchange), the norm's sum is a shuffle tree, and a CTA loads several heads
// before it uses the first.  The angles of a CTA's tokens are computed once
// and shared by all their heads.  An angle is p f / pi in 64 bits, reduced to
// [-1, 1] before sincospi in 32: a 32-bit product would be wrong in the second
// digit at positions near 10^6.  All arithmetic on values is fp32; each output
// is rounded to bf16 once.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_internal.h"

namespace lb {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTb = 8;       // tokens of a CTA's block
constexpr int kUnroll = 3;      // heads a lane group loads before it uses the first

struct HeadsParams {
    HeadGroup g[kMaxHeadGroups];
    int first[kMaxHeadGroups + 1];  // forward: first head of each group; backward: first CTA
    int ngroups;
    int tokens, d, rd, tb;
    const int32_t *positions;
    const float *inv_freq;
    float eps;
    float *part;  // backward: dw partials [CTA][d]
};

struct Vals {
    float v[8];
};

// The 8 elements of a head that `lane` of L holds: PAIRS (or past the rotated
// part): 8 lane ..; halves: 4 lane .. and rd/2 + 4 lane ..
template <bool PAIRS>
__device__ __forceinline__ void element_offsets(int lane, int rd, int &e0, int &e1)
{
    e0 = 8 * lane;
    e1 = e0 + 4;
    if (!PAIRS && 8 * lane < rd) {
        e0 = 4 * lane;
        e1 = (rd >> 1) + 4 * lane;
    }
}

__device__ __forceinline__ void load8(const uint16_t *p, int e0, int e1, uint2 &a, uint2 &b)
{
    a = *reinterpret_cast<const uint2 *>(p + e0);
    b = *reinterpret_cast<const uint2 *>(p + e1);
}

__device__ __forceinline__ Vals unpack8(const uint2 &a, const uint2 &b)
{
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
    Vals r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.v[2 * i] = __uint_as_float(w[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return r;
}

__device__ __forceinline__ void store8(uint16_t *p, int e0, int e1, const Vals &r)
{
    *reinterpret_cast<uint2 *>(p + e0) = make_uint2(pack_bf162(r.v[0], r.v[1]), pack_bf162(r.v[2], r.v[3]));
    *reinterpret_cast<uint2 *>(p + e1) = make_uint2(pack_bf162(r.v[4], r.v[5]), pack_bf162(r.v[6], r.v[7]));
}

template <int L>
__device__ __forceinline__ float group_sum(float s)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Rotates a lane's elements in place by the angles (cos, sin) of its pairs;
// sgn = -1 is the transpose.  `cs`: this token's [rd / 2].
template <bool PAIRS>
__device__ __forceinline__ void rotate8(Vals &r, const float2 *cs, int lane, float sgn)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = PAIRS ? 2 * i : i, b = PAIRS ? 2 * i + 1 : i + 4;
        const float2 t = cs[4 * lane + i];
        const float sn = sgn * t.y;
        const float x = r.v[a], y = r.v[b];
        r.v[a] = x * t.x - y * sn;
        r.v[b] = y * t.x + x * sn;
    }
}

// cos and sin of the angles of tokens t0 .. t0 + nt - 1 into cs [nt][rd / 2].
__device__ __forceinline__ void fill_angles(const HeadsParams &p, int t0, int nt, float2 *cs)
{
    const int half = p.rd >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int tok = i / half;
        const double turns = (double)__ldg(p.positions + t0 + tok) * (double)__ldg(p.inv_freq + (i - tok * half)) *
                             0.31830988618379067154;  // angle / pi
        float s, c;
        sincospif((float)(turns - 2.0 * rint(0.5 * turns)), &s, &c);
        cs[i] = make_float2(c, s);
    }
}

// One CTA per block of tb tokens; its lane groups take the block's heads (of
// every tensor, tokens outermost) in turn.
template <int L, bool PAIRS>
__global__ void __launch_bounds__(kThreads) heads_forward_kernel(const __grid_constant__ HeadsParams p)
{
    constexpr int kSlots = kThreads / L;
    __shared__ float2 cs[kMaxTb * 128];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const int t0 = blockIdx.x * p.tb, nt = min(p.tb, p.tokens - t0);
    const int heads = p.first[p.ngroups], rows = nt * heads;
    const bool on = 8 * lane < p.d;
    const int ln = on ? lane : 0;  // lanes past a narrow head stay in the shuffles
    int e0, e1;
    element_offsets<PAIRS>(ln, p.rd, e0, e1);
    const int half = p.rd >> 1;
    fill_angles(p, t0, nt, cs);  // positions and frequencies come before the kernels this one waits for
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    for (int r0 = slot; r0 - slot < rows; r0 += kSlots * kUnroll) {
        uint2 a[kUnroll], b[kUnroll];
        int64_t off[kUnroll];
        int tok[kUnroll], gi[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = min(r0 + u * kSlots, rows - 1);
            tok[u] = r / heads;
            const int h = r - tok[u] * heads;
            int g = 0;
            while (g + 1 < p.ngroups && h >= p.first[g + 1]) ++g;
            gi[u] = g;
            off[u] = (int64_t)(h - p.first[g]) * p.d;
            load8(p.g[g].in + (int64_t)(t0 + tok[u]) * p.g[g].ld_in + off[u], e0, e1, a[u], b[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const HeadGroup &G = p.g[gi[u]];
            Vals x = unpack8(a[u], b[u]);
            if (G.weight != nullptr || L < 32) {  // a warp's slots may hold heads of different tensors
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x.v[i] * x.v[i];
                s = group_sum<L>(on ? s : 0.0f);
                if (G.weight != nullptr) {
                    const float rstd = rsqrtf(s / (float)p.d + p.eps);
                    uint2 wa, wb;
                    load8(G.weight, e0, e1, wa, wb);
                    const Vals w = unpack8(wa, wb);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x.v[i] = x.v[i] * rstd * w.v[i];
                }
            }
            if (8 * ln < p.rd) rotate8<PAIRS>(x, cs + tok[u] * half, ln, 1.0f);
            if (on && r0 + u * kSlots < rows)
                store8(G.out + (int64_t)(t0 + tok[u]) * G.ld_out + off[u], e0, e1, x);
        }
    }
}

// CTAs first[g] .. first[g + 1] - 1 take tensor g; each walks over blocks of
// tb tokens and keeps its lanes' part of dw in registers.
template <int L, bool PAIRS>
__global__ void __launch_bounds__(kThreads) heads_backward_kernel(const __grid_constant__ HeadsParams p)
{
    constexpr int kSlots = kThreads / L;
    __shared__ float2 cs[2][kMaxTb * 128];
    __shared__ float red[kSlots * 8 * L];
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    int g = 0;
    while (g + 1 < p.ngroups && (int)blockIdx.x >= p.first[g + 1]) ++g;
    const HeadGroup &G = p.g[g];
    const int cta = blockIdx.x - p.first[g], ctas = p.first[g + 1] - p.first[g];
    const bool on = 8 * lane < p.d;
    const int ln = on ? lane : 0;
    int e0, e1;
    element_offsets<PAIRS>(ln, p.rd, e0, e1);
    const int half = p.rd >> 1, heads = G.heads;
    const bool norm = G.weight != nullptr;
    Vals w, acc;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc.v[i] = 0.0f, w.v[i] = 1.0f;
    if (norm) {
        uint2 wa, wb;
        load8(G.weight, e0, e1, wa, wb);
        w = unpack8(wa, wb);
    }
    pdl_wait();
    pdl_launch_dependents();
    const int blocks = (p.tokens + p.tb - 1) / p.tb;
    int buf = 0;
    for (int blk = cta; blk < blocks; blk += ctas, buf ^= 1) {
        const int t0 = blk * p.tb, nt = min(p.tb, p.tokens - t0), rows = nt * heads;
        fill_angles(p, t0, nt, cs[buf]);
        __syncthreads();  // one barrier a block: the other buffer's readers passed the barrier before it
        for (int r0 = slot; r0 - slot < rows; r0 += kSlots * kUnroll) {
            uint2 xa[kUnroll], xb[kUnroll], da[kUnroll], db[kUnroll];
            int64_t off[kUnroll];
            int tok[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int r = min(r0 + u * kSlots, rows - 1);
                tok[u] = r / heads;
                off[u] = (int64_t)(r - tok[u] * heads) * p.d;
                const int64_t t = t0 + tok[u];
                load8(G.dout + t * G.ld_dout + off[u], e0, e1, da[u], db[u]);
                if (norm) load8(G.in + t * G.ld_in + off[u], e0, e1, xa[u], xb[u]);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const bool live = on && r0 + u * kSlots < rows;
                Vals dn = unpack8(da[u], db[u]);
                if (8 * ln < p.rd) rotate8<PAIRS>(dn, cs[buf] + tok[u] * half, ln, -1.0f);
                if (norm) {  // uniform over the CTA
                    Vals x = unpack8(xa[u], xb[u]);
                    float ss = 0.0f, sd = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        ss += x.v[i] * x.v[i];
                        sd += w.v[i] * dn.v[i] * x.v[i];
                    }
                    ss = group_sum<L>(on ? ss : 0.0f);
                    sd = group_sum<L>(on ? sd : 0.0f);
                    const float rstd = rsqrtf(ss / (float)p.d + p.eps);
                    const float c = sd * rstd / (float)p.d;  // mean(w dn x^)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = x.v[i] * rstd;
                        if (live) acc.v[i] += dn.v[i] * xh;
                        dn.v[i] = rstd * (w.v[i] * dn.v[i] - xh * c);
                    }
                }
                if (live) store8(G.out + (int64_t)(t0 + tok[u]) * G.ld_out + off[u], e0, e1, dn);
            }
        }
    }
    if (G.dweight == nullptr) return;  // uniform over the CTA
    // this CTA's dw: the slots in order
    if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            red[slot * p.d + e0 + i] = acc.v[i];
            red[slot * p.d + e1 + i] = acc.v[4 + i];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.d; e += kThreads) {
        float s = 0.0f;
        for (int q = 0; q < kSlots; ++q) s += red[q * p.d + e];
        p.part[(int64_t)blockIdx.x * p.d + e] = s;
    }
}

// dweight of tensor blockIdx.y: its CTAs' partial rows, 32 columns a CTA; warp
// q adds rows q, q + 8, ... and warp 0 the eight sums, always in that order.
__global__ void __launch_bounds__(256) heads_dweight_kernel(const __grid_constant__ HeadsParams p)
{
    __shared__ float sums[8][32];
    const HeadGroup &G = p.g[blockIdx.y];
    if (G.dweight == nullptr) {
        pdl_wait();
        return;
    }
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    pdl_wait();
    float s = 0.0f;
    if (e < p.d)
        for (int r = p.first[blockIdx.y] + q; r < p.first[blockIdx.y + 1]; r += 8) s += p.part[(int64_t)r * p.d + e];
    sums[q][lane] = s;
    __syncthreads();
    if (q == 0 && e < p.d) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sums[i][lane];
        G.dweight[e] = t;
    }
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, const HeadsParams &p, cudaStream_t stream)
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

HeadsParams make_params(const HeadsArgs &a)
{
    HeadsParams p{};
    for (int g = 0; g < a.ngroups; ++g) p.g[g] = a.group[g];
    p.ngroups = a.ngroups;
    p.tokens = a.tokens;
    p.d = a.head_dim;
    p.rd = a.rotary_dim;
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.eps = a.eps;
    return p;
}

int lanes_of(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : 32; }

}  // namespace

size_t heads_backward_workspace_bytes(int head_dim) { return sizeof(float) * (size_t)kMaxHeadCtas * (size_t)head_dim; }

cudaError_t heads_forward(const HeadsArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    HeadsParams p = make_params(a);
    for (int g = 0; g < a.ngroups; ++g) p.first[g + 1] = p.first[g] + a.group[g].heads;
    const int heads = p.first[a.ngroups], L = lanes_of(a.head_dim), slots = kThreads / L;
    // tokens a CTA: enough rows for every lane group to load kUnroll heads at
    // once, while that leaves a CTA for every SM
    p.tb = std::max(1, std::min({kMaxTb, slots * kUnroll / heads, a.tokens / dev.sm_count}));
    const dim3 grid((unsigned)((a.tokens + p.tb - 1) / p.tb));
    const bool pairs = a.pairs != 0;
    if (L == 8)
        return pairs ? launch_pdl(heads_forward_kernel<8, true>, grid, p, stream)
                     : launch_pdl(heads_forward_kernel<8, false>, grid, p, stream);
    if (L == 16)
        return pairs ? launch_pdl(heads_forward_kernel<16, true>, grid, p, stream)
                     : launch_pdl(heads_forward_kernel<16, false>, grid, p, stream);
    return pairs ? launch_pdl(heads_forward_kernel<32, true>, grid, p, stream)
                 : launch_pdl(heads_forward_kernel<32, false>, grid, p, stream);
}

cudaError_t heads_backward(const HeadsArgs &a, float *workspace, const DeviceInfo &dev, cudaStream_t stream)
{
    HeadsParams p = make_params(a);
    p.part = workspace;
    const int L = lanes_of(a.head_dim), slots = kThreads / L;
    int heads = 0, fewest = 1 << 30;
    bool any = false;
    for (int g = 0; g < a.ngroups; ++g) {
        heads += a.group[g].heads;
        fewest = std::min(fewest, a.group[g].heads);
        any = any || a.group[g].dweight != nullptr;
    }
    p.tb = std::max(1, std::min({kMaxTb, slots * kUnroll / fewest, a.tokens / dev.sm_count}));
    const int blocks = (a.tokens + p.tb - 1) / p.tb;
    // about four CTAs an SM, shared out by the tensors' heads
    const int total = std::min(kMaxHeadCtas - kMaxHeadGroups, 4 * dev.sm_count);
    for (int g = 0; g < a.ngroups; ++g) {
        const int n = (int)((int64_t)total * a.group[g].heads / heads);
        p.first[g + 1] = p.first[g] + std::max(1, std::min(n, blocks));
    }
    const dim3 grid((unsigned)p.first[a.ngroups]);
    const bool pairs = a.pairs != 0;
    cudaError_t e;
    if (L == 8)
        e = pairs ? launch_pdl(heads_backward_kernel<8, true>, grid, p, stream)
                  : launch_pdl(heads_backward_kernel<8, false>, grid, p, stream);
    else if (L == 16)
        e = pairs ? launch_pdl(heads_backward_kernel<16, true>, grid, p, stream)
                  : launch_pdl(heads_backward_kernel<16, false>, grid, p, stream);
    else
        e = pairs ? launch_pdl(heads_backward_kernel<32, true>, grid, p, stream)
                  : launch_pdl(heads_backward_kernel<32, false>, grid, p, stream);
    if (e != cudaSuccess || !any) return e;
    return launch_pdl(heads_dweight_kernel, dim3((unsigned)((a.head_dim + 31) / 32), (unsigned)a.ngroups), p, stream);
}

}  // namespace lb
