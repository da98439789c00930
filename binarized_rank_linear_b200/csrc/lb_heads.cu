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
// bounds both passes: 4 bytes an element forward, 6 backward.  What costs next
// is instructions, and keeping enough bytes under way without them: one thread
// brings the heads of the next tokens to shared memory by bulk copies, kStages
// ahead, two warps compute those tokens' angles, once for all their heads, and
// the other warps take token after token, a few lanes to a head with both ends
// of a rotated pair in the same lane (so the rotation needs no exchange, and the
// norm's sum is a shuffle tree), the head's weights in registers, 16 elements a
// lane where the sizes allow it, else 8.  For 8192 tokens of 40 + 8 heads of
// 128: 36 us forward (5.6 TB/s), 62 us backward (4.9 TB/s).  (A CTA a token: 63 us
// forward; CTAs that stay, with the next tokens in registers, 41 us forward and 86
// us backward; 8 elements a lane on twice the threads, 67 us backward, 16 on twice
// the threads 74.)
// An angle is p f / pi in 64 bits, reduced to [-1, 1] before sincospi in 32: a
// 32-bit product would be wrong in the second digit at positions near 10^6.
// All arithmetic on values is fp32; each output is rounded to bf16 once.
#include <algorithm>
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_operators.h"
#include "lb_tc.cuh"

namespace lb {
namespace {

using namespace tc;

constexpr int kMaxCompute = 384;  // threads that have a head
constexpr int kAngleWarps = 2;
constexpr int kStages = 4;
constexpr int kAngles = 1024;     // most angles of a stage

struct HeadsParams {
    HeadGroup g[kMaxHeadGroups];
    int first[kMaxHeadGroups + 1];  // first head of each tensor
    int ngroups;
    int tokens, d, rd;
    int tb;        // tokens of a stage: more than one where they have few heads
    int chunk;     // heads of a CTA (grid.y chunks of them)
    int warps;     // that have heads
    int row_bytes, stage_bytes;  // a token's heads of one tensor kind (input, or dout); a stage
    const int32_t *positions;
    const float *inv_freq;
    float eps;
    float *part;  // backward: dw partials [CTA][tensor][d]
    int *status;
};

// A lane's E elements of a head as rotated pairs (a[i], b[i]).  They lie in two
// runs of E / 2: with halves the a and the b, with neighbours as pairs (and past
// the rotated part) the first and the last of the pairs.
template <int E>
struct Vals {
    float a[E / 2], b[E / 2];
};
template <int E>
struct Run {
    uint32_t w[E / 4];
};
template <int E>
__device__ __forceinline__ Run<E> load_run(const uint16_t *p)
{
    Run<E> r;
    if constexpr (E == 16)
        *reinterpret_cast<uint4 *>(r.w) = *reinterpret_cast<const uint4 *>(p);
    else
        *reinterpret_cast<uint2 *>(r.w) = *reinterpret_cast<const uint2 *>(p);
    return r;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <int E, bool PAIRS>
__device__ __forceinline__ Vals<E> unpack(const Run<E> &x, const Run<E> &y)
{
    Vals<E> v;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        if (PAIRS) {
            v.a[i] = lo_of(x.w[i]);
            v.b[i] = hi_of(x.w[i]);
            v.a[E / 4 + i] = lo_of(y.w[i]);
            v.b[E / 4 + i] = hi_of(y.w[i]);
        } else {
            v.a[2 * i] = lo_of(x.w[i]);
            v.a[2 * i + 1] = hi_of(x.w[i]);
            v.b[2 * i] = lo_of(y.w[i]);
            v.b[2 * i + 1] = hi_of(y.w[i]);
        }
    }
    return v;
}
template <int E, bool PAIRS>
__device__ __forceinline__ void store(uint16_t *p, int gap, const Vals<E> &v)
{
    Run<E> x, y;
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
        x.w[i] = PAIRS ? pack_bf162(v.a[i], v.b[i]) : pack_bf162(v.a[2 * i], v.a[2 * i + 1]);
        y.w[i] = PAIRS ? pack_bf162(v.a[E / 4 + i], v.b[E / 4 + i]) : pack_bf162(v.b[2 * i], v.b[2 * i + 1]);
    }
    if constexpr (E == 16) {
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(x.w);
        *reinterpret_cast<uint4 *>(p + gap) = *reinterpret_cast<const uint4 *>(y.w);
    } else {
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(x.w);
        *reinterpret_cast<uint2 *>(p + gap) = *reinterpret_cast<const uint2 *>(y.w);
    }
}
// Where in the head pair i's a and b are, for a lane whose runs begin at e0 and e1.
template <int E, bool PAIRS>
__device__ __forceinline__ int place(int e0, int e1, int i, bool b)
{
    if (PAIRS) return (i < E / 4 ? e0 : e1) + 2 * (i % (E / 4)) + b;
    return (b ? e1 : e0) + i;
}

// Two fp32 operations in one instruction, on neighbours of an array.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair_of(const float *v)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v[0]), "f"(v[1]));
    return r;
}
__device__ __forceinline__ f32x2 both(float v)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void put_pair(float *v, f32x2 p) { asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(p)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <int E>
__device__ __forceinline__ float dot(const Vals<E> &x, const Vals<E> &y)
{
    f32x2 s = mul2(pair_of(x.a), pair_of(y.a)), t = mul2(pair_of(x.b), pair_of(y.b));
#pragma unroll
    for (int i = 2; i < E / 2; i += 2) {
        s = fma2(pair_of(x.a + i), pair_of(y.a + i), s);
        t = fma2(pair_of(x.b + i), pair_of(y.b + i), t);
    }
    float f[4];
    put_pair(f, s);
    put_pair(f + 2, t);
    return (f[0] + f[1]) + (f[2] + f[3]);
}
template <int L>
__device__ __forceinline__ float group_sum(float s)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Bulk copy of `bytes` (a multiple of 16) to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
template <int E>
__device__ __forceinline__ Run<E> shared_run(uint32_t at)
{
    Run<E> r;
    if constexpr (E == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                     : "r"(at)
                     : "memory");
    else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(at) : "memory");
    return r;
}

// Rotates a lane's pairs by the angles from `cos` and `sin` on, or back.
template <int E, bool BACK>
__device__ __forceinline__ void rotate(Vals<E> &v, const float *cos, const float *sin)
{
#pragma unroll
    for (int i = 0; i < E / 2; i += 4) {
        const float4 c4 = *reinterpret_cast<const float4 *>(cos + i), s4 = *reinterpret_cast<const float4 *>(sin + i);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v.a[i + j], y = v.b[i + j];
            v.a[i + j] = BACK ? fmaf(y, s[j], x * c[j]) : fmaf(-y, s[j], x * c[j]);
            v.b[i + j] = BACK ? fmaf(-x, s[j], y * c[j]) : fmaf(x, s[j], y * c[j]);
        }
    }
}

// CTA (x, y): stages x, x + gridDim.x, ... of p.tb tokens, heads of chunk y.
// Warps 0 .. p.warps - 1 have heads, L lanes each one of one token of a stage;
// then the copying warp, then the angles'.
template <int L, int E, bool PAIRS, bool BACK>
__global__ void __launch_bounds__(kMaxCompute + 32 * (1 + kAngleWarps), BACK ? 1 : 2)
    heads_kernel(const __grid_constant__ HeadsParams p)
{
    extern __shared__ __align__(128) uint8_t shared[];
    __shared__ alignas(8) unsigned long long bars[2 * kStages];
    __shared__ int abort_shared;
    volatile int &abort_flag = abort_shared;
    const int warp = threadIdx.x >> 5, half = p.rd >> 1, tokens = p.tokens, tb = p.tb;
    const int heads = p.first[p.ngroups], h0 = blockIdx.y * p.chunk, nh = min(p.chunk, heads - h0);
    const uint32_t base = smem_u32(shared), full0 = smem_u32(bars), empty0 = full0 + 8 * kStages;
    float *angles = reinterpret_cast<float *>(shared + kStages * p.stage_bytes);  // [stage][cos, sin][tb][half]
    const int room = tb * half, stride = gridDim.x * tb, t0 = blockIdx.x * tb;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full0 + 8 * s, 1 + (half > 0 ? kAngleWarps : 0));
            mbar_init(empty0 + 8 * s, p.warps);
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // Every role waits for the work ahead on the stream, which may have let this
    // launch start early: it may be what writes positions or a weight, and the
    // bounded waits below must not count the time that it takes.  (Angles ahead of
    // the wait took up to 1 us less behind a projection with adapters, 4 tokens.)
    pdl_wait();
    pdl_launch_dependents();
    if (warp == p.warps) {
        if ((threadIdx.x & 31) == 0) {
            int s = 0;
            uint32_t ph = 1;
            for (int t = t0; t < tokens; t += stride) {
                if (!mbar_wait(empty0 + 8 * s, ph) || abort_flag) {
                    abort_flag = 1;
                    break;
                }
                const int n = min(tb, tokens - t);
                const uint32_t bar = full0 + 8 * s, dst = base + s * p.stage_bytes;
                uint32_t tx = 0;
                for (int g = 0; g < p.ngroups; ++g) {
                    const int a = max(p.first[g], h0), b = min(p.first[g + 1], h0 + nh);
                    if (a < b) tx += (uint32_t)(n * (b - a) * p.d * 2) * (!BACK ? 1u : p.g[g].weight != nullptr ? 2u : 1u);
                }
                mbar_arrive_expect_tx(bar, tx);
                for (int g = 0; g < p.ngroups; ++g) {
                    const HeadGroup &G = p.g[g];
                    const int a = max(p.first[g], h0), b = min(p.first[g + 1], h0 + nh);
                    if (a >= b) continue;
                    const uint32_t bytes = (uint32_t)((b - a) * p.d * 2), at = dst + (uint32_t)((a - h0) * p.d * 2);
                    const int64_t off = (int64_t)(a - p.first[g]) * p.d;
                    for (int k = 0; k < n; ++k) {
                        if (!BACK || G.weight != nullptr)
                            bulk_load(at + k * p.row_bytes, G.in + (int64_t)(t + k) * G.ld_in + off, bytes, bar);
                        if (BACK)
                            bulk_load(at + (tb + k) * p.row_bytes, G.dout + (int64_t)(t + k) * G.ld_dout + off, bytes, bar);
                    }
                }
                if (++s == kStages) s = 0, ph ^= 1;
            }
            if (abort_flag) {  // copies in flight land within microseconds
                const unsigned long long since = globaltimer();
                while (globaltimer() - since < 200000ull) {
                }
            }
        }
    } else if (warp > p.warps) {
        const int tid = threadIdx.x - 32 * (p.warps + 1);
        int s = 0;
        uint32_t ph = 1;
        for (int t = t0; half > 0 && t < tokens; t += stride) {
            const bool ok = mbar_wait(empty0 + 8 * s, ph) && !abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            float *cos = angles + 2 * s * room, *sin = cos + room;
            const int n = min(tb, tokens - t) * half;
            for (int i = tid; i < n; i += 32 * kAngleWarps) {
                const int tok = i / half;
                const double turns = (double)__ldcg(p.positions + t + tok) * (double)__ldcg(p.inv_freq + (i - tok * half)) *
                                     0.31830988618379067154;  // angle / pi
                sincospif((float)(turns - 2.0 * rint(0.5 * turns)), sin + i, cos + i);
            }
            __syncwarp();
            if ((tid & 31) == 0) mbar_arrive(full0 + 8 * s);
            if (++s == kStages) s = 0, ph ^= 1;
        }
    }
    const int lane = threadIdx.x % L, slot = threadIdx.x / L;
    const bool in_head = E * lane < p.d;
    const int ln = in_head ? lane : 0;  // lanes past a narrow head stay in the shuffles
    const bool turned = E * ln < p.rd;
    const int e0 = !PAIRS && turned ? E / 2 * ln : E * ln, gap = !PAIRS && turned ? half : E / 2;
    Vals<E> acc;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) acc.a[i] = acc.b[i] = 0.0f;
    if (warp < p.warps) {
        const float inv_d = 1.0f / (float)p.d, eps = p.eps;
        // this lane group's token within a stage (past every token where it has no head) and head
        const bool on = slot < tb * nh;
        const int off = on ? slot / nh : tokens, h = h0 + (on ? slot - off * nh : 0);
        int g = 0;
        while (g + 1 < p.ngroups && h >= p.first[g + 1]) ++g;
        const HeadGroup &G = p.g[g];
        const bool norm = G.weight != nullptr, live0 = on && in_head;
        const int64_t step = (int64_t)stride * G.ld_out;
        uint16_t *out = G.out + (int64_t)(h - p.first[g]) * p.d + e0 + (on ? (int64_t)(t0 + off) * G.ld_out : 0);
        Run<E> w0{}, w1{};
        if (norm) {
            w0 = load_run<E>(G.weight + e0);
            w1 = load_run<E>(G.weight + e0 + gap);
        }
        const Vals<E> w = unpack<E, PAIRS>(w0, w1);
        const bool any_norm = __any_sync(0xffffffffu, norm);
        const uint32_t mine = base + (uint32_t)((on ? off : 0) * p.row_bytes + ((h - h0) * p.d + e0) * 2), gap2 = 2 * gap;
        const uint32_t douts = (uint32_t)(tb * p.row_bytes), stage_bytes = p.stage_bytes;
        const float *cos0 = angles + (on ? off : 0) * half + E / 2 * ln;
        int s = 0, left = on ? tokens - off : 0;  // tokens from this group's on
        uint32_t ph = 0;
        for (int t = t0; t < tokens; t += stride) {
            const bool ok = mbar_wait(full0 + 8 * s, ph) && !abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            const uint32_t at = mine + s * stage_bytes;
            const float *cos = cos0 + 2 * s * room, *sin = cos + room;
            const bool live = live0 && t < left;
            if (!BACK) {
                Vals<E> x = unpack<E, PAIRS>(shared_run<E>(at), shared_run<E>(at + gap2));
                if (any_norm) {
                    const float q = group_sum<L>(in_head ? dot(x, x) : 0.0f);
                    const float rstd = rsqrtf(fmaf(q, inv_d, eps));
                    if (norm) {
                        const f32x2 r2 = both(rstd);
#pragma unroll
                        for (int i = 0; i < E / 2; i += 2) {
                            put_pair(x.a + i, mul2(pair_of(x.a + i), mul2(r2, pair_of(w.a + i))));
                            put_pair(x.b + i, mul2(pair_of(x.b + i), mul2(r2, pair_of(w.b + i))));
                        }
                    }
                }
                if (turned) rotate<E, false>(x, cos, sin);
                __syncwarp();
                if ((threadIdx.x & 31) == 0) mbar_arrive(empty0 + 8 * s);
                if (live) store<E, PAIRS>(out, gap, x);
            } else {
                Vals<E> dn = unpack<E, PAIRS>(shared_run<E>(at + douts), shared_run<E>(at + douts + gap2));
                if (turned) rotate<E, true>(dn, cos, sin);
                if (any_norm) {
                    const Vals<E> x = unpack<E, PAIRS>(shared_run<E>(at), shared_run<E>(at + gap2));
                    __syncwarp();
                    if ((threadIdx.x & 31) == 0) mbar_arrive(empty0 + 8 * s);
                    Vals<E> wd;
#pragma unroll
                    for (int i = 0; i < E / 2; i += 2) {
                        put_pair(wd.a + i, mul2(pair_of(w.a + i), pair_of(dn.a + i)));
                        put_pair(wd.b + i, mul2(pair_of(w.b + i), pair_of(dn.b + i)));
                    }
                    const float ss = group_sum<L>(in_head ? dot(x, x) : 0.0f);
                    const float sd = group_sum<L>(in_head ? dot(wd, x) : 0.0f);
                    const float rstd = rsqrtf(fmaf(ss, inv_d, eps));
                    const float c = -sd * rstd * inv_d;  // - mean(w dn x^)
                    if (norm) {
                        const f32x2 r2 = both(rstd), c2 = both(c);
#pragma unroll
                        for (int i = 0; i < E / 2; i += 2) {
                            const f32x2 ha = mul2(pair_of(x.a + i), r2), hb = mul2(pair_of(x.b + i), r2);  // x^
                            if (live) {
                                put_pair(acc.a + i, fma2(pair_of(dn.a + i), ha, pair_of(acc.a + i)));
                                put_pair(acc.b + i, fma2(pair_of(dn.b + i), hb, pair_of(acc.b + i)));
                            }
                            put_pair(dn.a + i, mul2(r2, fma2(ha, c2, pair_of(wd.a + i))));
                            put_pair(dn.b + i, mul2(r2, fma2(hb, c2, pair_of(wd.b + i))));
                        }
                    }
                } else {
                    __syncwarp();
                    if ((threadIdx.x & 31) == 0) mbar_arrive(empty0 + 8 * s);
                }
                if (live) store<E, PAIRS>(out, gap, dn);
            }
            out += step;
            if (++s == kStages) s = 0, ph ^= 1;
        }
    }
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) set_status(p.status, LB_ERR_DEVICE_TIMEOUT);
    if (!BACK || p.part == nullptr) return;
    // this CTA's dw of each tensor: the lane groups' in order, where the stages were
    float *red = reinterpret_cast<float *>(shared);
    if (slot < tb * nh && in_head) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            red[slot * p.d + place<E, PAIRS>(e0, e0 + gap, i, false)] = acc.a[i];
            red[slot * p.d + place<E, PAIRS>(e0, e0 + gap, i, true)] = acc.b[i];
        }
    }
    __syncthreads();
    const int64_t cta = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (int i = threadIdx.x; i < p.ngroups * p.d; i += (int)blockDim.x) {
        const int q = i / p.d, e = i - q * p.d;
        float s = 0.0f;
        for (int k = 0; k < tb; ++k)
            for (int j = max(p.first[q], h0); j < min(p.first[q + 1], h0 + nh); ++j) s += red[(k * nh + j - h0) * p.d + e];
        p.part[cta * p.ngroups * p.d + i] = s;
    }
}

// dweight of tensor blockIdx.y: its partials of all `ctas`, 32 columns a CTA; warp
// q adds CTAs q, q + 8, ... and warp 0 the eight sums, always in that order.
__global__ void __launch_bounds__(256) heads_dweight_kernel(const __grid_constant__ HeadsParams p, int ctas)
{
    __shared__ float sums[8][32];
    const HeadGroup &G = p.g[blockIdx.y];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane;
    pdl_wait();
    if (G.dweight == nullptr) return;
    float s = 0.0f;
    if (e < p.d)
#pragma unroll 4
        for (int r = q; r < ctas; r += 8) s += p.part[((int64_t)r * p.ngroups + blockIdx.y) * p.d + e];
    sums[q][lane] = s;
    __syncthreads();
    if (q == 0 && e < p.d) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sums[i][lane];
        G.dweight[e] = t;
    }
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs of a heads launch: chunks of heads, and for each as many CTAs as the
// device runs at once, or as there are stages.
template <int L, int E, bool BACK>
cudaError_t launch_heads(const HeadsArgs &a, HeadsParams &p, const DeviceInfo &dev, cudaStream_t stream, int *ctas)
{
    const int heads = p.first[a.ngroups], slots = kMaxCompute / L;
    const int chunks = (heads + slots - 1) / slots;
    p.chunk = (heads + chunks - 1) / chunks;
    // tokens of a stage, while every SM still has one
    const int per_sm = std::max(1, a.tokens / dev.sm_count), half = std::max(1, a.rotary_dim / 2);
    p.tb = std::max(1, std::min({slots / p.chunk, per_sm, kAngles / half}));
    p.warps = (p.tb * p.chunk * L + 31) / 32;
    p.row_bytes = p.chunk * a.head_dim * 2;
    p.stage_bytes = ((BACK ? 2 : 1) * p.tb * p.row_bytes + 127) & ~127;
    p.status = dev.status;
    const size_t smem = (size_t)kStages * ((size_t)p.stage_bytes + sizeof(float) * (size_t)(p.tb * a.rotary_dim));
    const int stages = (a.tokens + p.tb - 1) / p.tb;
    dim3 grid((unsigned)std::min(stages, std::max(1, (BACK ? 1 : 2) * dev.sm_count / chunks)), (unsigned)chunks);
    if (BACK) grid.x = std::min(grid.x, (unsigned)std::max(1, kMaxHeadCtas / chunks));
    *ctas = (int)(grid.x * grid.y);
    const int threads = 32 * (p.warps + 1 + kAngleWarps);
    return a.pairs ? launch_pdl(heads_kernel<L, E, true, BACK>, grid, threads, smem, stream, p)
                   : launch_pdl(heads_kernel<L, E, false, BACK>, grid, threads, smem, stream, p);
}

template <bool BACK>
cudaError_t dispatch_heads(const HeadsArgs &a, HeadsParams &p, const DeviceInfo &dev, cudaStream_t stream, int *ctas)
{
    for (int g = 0; g < a.ngroups; ++g) {
        p.g[g] = a.group[g];
        p.first[g + 1] = p.first[g] + a.group[g].heads;
    }
    p.ngroups = a.ngroups;
    p.tokens = a.tokens;
    p.d = a.head_dim;
    p.rd = a.rotary_dim;
    p.positions = a.positions;
    p.inv_freq = a.inv_freq;
    p.eps = a.eps;
    const int d = a.head_dim;
    if (d % 16 == 0 && a.rotary_dim % 16 == 0)
        return d <= 64    ? launch_heads<4, 16, BACK>(a, p, dev, stream, ctas)
               : d <= 128 ? launch_heads<8, 16, BACK>(a, p, dev, stream, ctas)
                          : launch_heads<16, 16, BACK>(a, p, dev, stream, ctas);
    return d <= 64    ? launch_heads<8, 8, BACK>(a, p, dev, stream, ctas)
           : d <= 128 ? launch_heads<16, 8, BACK>(a, p, dev, stream, ctas)
                      : launch_heads<32, 8, BACK>(a, p, dev, stream, ctas);
}

}  // namespace

// A row of dw partials for each tensor of every CTA.  A chunk has room for
// kMaxCompute / 32 heads at least, so the CTAs' rows do not run out of it.
static_assert((kMaxHeads + kMaxCompute / 32 - 1) / (kMaxCompute / 32) <= kMaxHeadCtas, "a CTA for each chunk of heads");
size_t heads_backward_workspace_bytes(int head_dim)
{
    return sizeof(float) * (size_t)kMaxHeadCtas * (size_t)kMaxHeadGroups * (size_t)head_dim;
}

cudaError_t heads_forward(const HeadsArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    HeadsParams p{};
    int ctas;
    return dispatch_heads<false>(a, p, dev, stream, &ctas);
}

cudaError_t heads_backward(const HeadsArgs &a, float *workspace, const DeviceInfo &dev, cudaStream_t stream)
{
    HeadsParams p{};
    bool any = false;
    for (int g = 0; g < a.ngroups; ++g) any = any || a.group[g].dweight != nullptr;
    p.part = any ? workspace : nullptr;
    int ctas;
    const cudaError_t e = dispatch_heads<true>(a, p, dev, stream, &ctas);
    if (e != cudaSuccess || !any) return e;
    return launch_pdl(heads_dweight_kernel, dim3((unsigned)((a.head_dim + 31) / 32), (unsigned)a.ngroups), 256, 0, stream, p, ctas);
}

cudaError_t heads_prepare_device(const DeviceInfo &dev)
{
    (void)dev;
    // stages of two tensors of kMaxCompute * 16 elements, and the angles
    const int bytes = kStages * (2 * kMaxCompute * 16 * 2 + 128 + 2 * kAngles * (int)sizeof(float));
    cudaError_t e = cudaSuccess;
    auto allow = [&](auto kernel) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    auto all = [&](auto l, auto n) {
        constexpr int L = decltype(l)::value, E = decltype(n)::value;
        allow(heads_kernel<L, E, false, false>);
        allow(heads_kernel<L, E, true, false>);
        allow(heads_kernel<L, E, false, true>);
        allow(heads_kernel<L, E, true, true>);
    };
    using std::integral_constant;
    all(integral_constant<int, 4>{}, integral_constant<int, 16>{});
    all(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    all(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    all(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    all(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    all(integral_constant<int, 32>{}, integral_constant<int, 8>{});
    return e;
}

}  // namespace lb
