// lb_adapters.cu - low-rank adapters of many requests beside a shared
// projection: the dispatch by token count and the kernels for small batches.
//
//     y[m] = base[m] + s_i B_i (A_i x[m]),  i = ids[m]
//
// At decode a batch reads the adapters its tokens use and little else: 2 r (n_in
// + n_out) bytes an adapter against 4 r (n_in + n_out) operations a token.  What
// counts is how few round trips to memory the two launches make:
//   shrink  a CTA takes up to kGroup tokens of one adapter, 16 rows of A and
//           1024 columns; a warp 128 of the columns; v partials
//           [slice][token][rank] in fp32
//   expand  a CTA takes the same tokens and 256 outputs, a warp 32 of them; the
//           slices are added in order, scaled, and split for the products
// The tokens are the 16 rows of register matrix products (m16n8k16) whose
// operands come straight from memory: which column is which k does not matter to
// a product as long as both operands agree, so a lane takes 16 bytes at once - 8
// columns of one row - and feeds them to two products.  Everything a CTA reads is
// asked for at once; expand asks for its weights and base while shrink still runs
// (programmatic dependent launch).  Tokens that share an adapter read its weights
// once per kGroup of them, wherever they stand in the batch.  Each CTA finds the
// groups for itself, once, and takes its units one after the other, the next one's
// weights asked for before the last is written; in expand a CTA's units are a run,
// so that v is put together once for many of them.
// Measured, both launches, operands not in L2, one pass behind the other: 1 token
// and three projections of 4096 x 4096, rank 16, 4.8 us; 100 tokens, 16 adapters of
// rank 32, 5120 to 2 x 17408 columns, 20.9 us, 2.9 TB/s (60 us with fp32 FMAs, a
// thread a row of B: most of it spent unpacking and on 16-byte pieces of 32 rows at
// a time; 36 us with the products but a CTA a unit: most of it spent finding
// groups, one wave of CTAs after the other; 1.4 us more with the units dealt out in
// turn); 128 tokens, 32 adapters of rank 128, 4096 x 4096, 22 us, 3.1 TB/s.  What is
// left is the chain of each unit: partials, split, product, store.
//
// For up to 128 + 48 tokens for each adapter of the pool, at most 512, or 24 for
// each, at most kAdapterSmallTokens (2048); beyond, and for the backward pass, the
// tcgen05 kernels of lb_adapters_mma.cu, whose tiles hold 128 tokens of one
// adapter: they pay where an adapter has many tokens.  The rule knows the tokens
// and the pool's size, which the host has; where the forms cross depends on rank
// and width too, and on how the tokens are spread, so that near its border it takes
// the slower form by up to 1.6 times.  Here and there (the small form with the
// groups found behind the wait, up to 3 us more than it takes now), tokens spread
// over the pool: 8 adapters of rank 16, 4096 x 4096, 256 tokens 9.7 and 18.6 us, 513
// tokens 13.5 and 19.3, 1024 tokens 19.6 and 23.7, 2048 tokens 32.6 and 29.3; 64 of
// rank 16, 5120 to 7168 columns, 1024 tokens 41 and 86, 1537 tokens 54 and 87; 32 of
// rank 128, 4096 x 4096, 768 tokens 43 and 42, 1024 tokens 51 and 44; 16 of rank 32,
// 5120 to 34816, 513 tokens 49 and 57, 768 tokens 65 and 58; 4 of rank 64, 4096 to
// 11008, 400 tokens 23 and 22, 513 tokens 28 and 24; 1 of rank 64, 4096 to 28672,
// 128 tokens 18.3 and 18.8, 200 tokens 24 and 21.  All tokens of one adapter of the
// 64: 512 tokens 18 and 21, 1536 tokens 41 and 30.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_operators.h"

namespace lb {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = 16;             // tokens of one adapter that a CTA takes together
constexpr int kRows = 16;              // rows of A of a shrink CTA
constexpr int kWarpCols = 128;         // columns of A of a shrink warp
constexpr int kSlice = kWarps * kWarpCols;
constexpr int kWarpOuts = 32;          // outputs of an expand warp
constexpr int kOutputs = kWarps * kWarpOuts;
constexpr int kShrinkCtas = 3;          // CTAs an SM: what their registers leave room for
constexpr int expand_ctas(int ks) { return ks < 2 ? 3 : 2; }
constexpr int kMostGroups = kAdapterSmallTokens / kGroup + LB_MAX_ADAPTERS + 1;
constexpr int kGroupBits = 12;         // of the sums over adapters: groups, and above them tokens
static_assert(kAdapterSmallTokens / kThreads * 32 <= 256 && LB_MAX_ADAPTER_RANK < 256 && LB_MAX_ADAPTERS < 32768 &&
                  kMostGroups < 1 << kGroupBits && kAdapterSmallTokens < 1 << 16,
              "8 bits hold a place among a warp's tokens and a rank, 16 an adapter and a token");
static_assert(kGroup * kRows == kThreads, "one thread for each partial of a shrink CTA");

struct SmallParams {
    const uint16_t *x;
    int64_t ldx;
    const int32_t *ids;
    int tokens, n_in, count, slices;
    AdapterProj proj[kMaxSiblings];
    float *part[kMaxSiblings];        // [slice][token][rank]
    int chunk0[kMaxSiblings + 1];     // expand: first chunk of kOutputs of each projection
    int row0[kMaxSiblings + 1];       // shrink: first kRows rows of each projection
    int nproj;
    int *status;
};

// The groups of a call: each adapter's tokens in order, cut every kGroup, adapter
// by adapter (those without one first).
struct Groups {
    uint16_t order[kAdapterSmallTokens];  // the tokens
    uint16_t start[kMostGroups];          // of each group in `order`
    int16_t ids[kMostGroups];             // -1: no adapter
    uint8_t size[kMostGroups];
    uint8_t rank[kMaxSiblings][kMostGroups];
};
// What finding them takes besides; a bin is an adapter's id + 1.
struct Finding {
    uint16_t count[LB_MAX_ADAPTERS + 1][kWarps];  // a warp's tokens of a bin, then where they begin in `order`
    uint16_t order0[LB_MAX_ADAPTERS + 2];         // of each bin
    uint16_t group0[LB_MAX_ADAPTERS + 1];
    uint16_t bin[kAdapterSmallTokens];            // of each token
    uint8_t place[kAdapterSmallTokens];           // among its warp's tokens of the bin
    uint32_t sums[kWarps];
};
// A token's adapter, -1 for none, and the rank of an adapter.
__device__ __forceinline__ int adapter_of(const SmallParams &p, int t)
{
    const int id = __ldcg(p.ids + t);
    return id >= p.count ? -1 : max(id, -1);
}
__device__ __forceinline__ uint8_t rank_of(const AdapterProj &P, int id)
{
    return (uint8_t)(id < 0 ? 0 : P.ranks == nullptr ? P.rank : max(0, min(P.rank, __ldcg(P.ranks + id))));
}
// Each warp takes a run of tokens, 32 at a time: those of one bin find each other
// (match), the table has how many came before them.
__device__ __forceinline__ int find_groups(const SmallParams &p, Groups &g, Finding &f)
{
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, bins = p.count + 1;
    auto id_of = [&](int t) { return adapter_of(p, t); };
    if (p.tokens == 1) {  // every thread has its id
        const int id = id_of(0);
        if (tid < p.nproj) g.rank[tid][0] = rank_of(p.proj[tid], id);
        if (tid == 0) {
            g.order[0] = g.start[0] = 0;
            g.ids[0] = (int16_t)id;
            g.size[0] = 1;
        }
        __syncthreads();
        return 1;
    }
    const int rounds = (p.tokens + kThreads - 1) / kThreads, t0 = w * rounds * 32 + lane;
#pragma unroll 1
    for (int b = tid; b < bins; b += kThreads) *reinterpret_cast<uint4 *>(f.count[b]) = make_uint4(0, 0, 0, 0);
    int bin = t0 < p.tokens ? id_of(t0) + 1 : -1;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
        const int t = t0 + 32 * i, next = t + 32 < p.tokens && i + 1 < rounds ? id_of(t + 32) + 1 : -1;
        const uint32_t peers = __match_any_sync(0xffffffffu, bin), earlier = peers & ((1u << lane) - 1u);
        const int had = bin >= 0 ? f.count[bin][w] : 0;
        __syncwarp();
        if (bin >= 0) {
            f.bin[t] = (uint16_t)bin;
            f.place[t] = (uint8_t)(had + __popc(earlier));
            if (earlier == 0) f.count[bin][w] = (uint16_t)(had + __popc(peers));
        }
        __syncwarp();
        bin = next;
    }
    __syncthreads();
    // a thread's bins, one after the other: their groups and tokens, summed over all
    const int per = (bins + kThreads - 1) / kThreads, b0 = min(tid * per, bins), b1 = min(b0 + per, bins);
    auto both = [&](int b) {
        const uint4 c = *reinterpret_cast<const uint4 *>(f.count[b]);
        const uint32_t h = (c.x & 0xffffu) + (c.x >> 16) + (c.y & 0xffffu) + (c.y >> 16) + (c.z & 0xffffu) + (c.z >> 16) +
                           (c.w & 0xffffu) + (c.w >> 16);
        return (h + kGroup - 1) / kGroup | h << kGroupBits;
    };
    uint32_t mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) mine += both(b);
    uint32_t at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t k = __shfl_up_sync(0xffffffffu, at, o);
        at += lane >= o ? k : 0;
    }
    if (lane == 31) f.sums[w] = at;
    __syncthreads();
    at -= mine;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        at += i < w ? f.sums[i] : 0;
        all += f.sums[i];
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const uint32_t n = both(b);
        f.group0[b] = (uint16_t)(at & ((1u << kGroupBits) - 1));
        uint32_t first = at >> kGroupBits;
        f.order0[b] = (uint16_t)first;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const uint32_t c = f.count[b][i];
            f.count[b][i] = (uint16_t)first;
            first += c;
        }
        at += n;
    }
    if (tid == 0) f.order0[bins] = (uint16_t)p.tokens;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
        const int t = t0 + 32 * i;
        if (t >= p.tokens) break;
        const int b = f.bin[t], to = f.count[b][w] + f.place[t], before = to - f.order0[b];
        g.order[to] = (uint16_t)t;
        if (before % kGroup == 0) {
            const int k = f.group0[b] + before / kGroup;
            g.start[k] = (uint16_t)to;
            g.ids[k] = (int16_t)(b - 1);
            g.size[k] = (uint8_t)min(kGroup, f.order0[b + 1] - to);
        }
    }
    __syncthreads();
    const int n = (int)(all & ((1u << kGroupBits) - 1));
#pragma unroll 1
    for (int i = tid; i < n * p.nproj; i += kThreads) {
        const int j = i / n, k = i - j * n;
        g.rank[j][k] = rank_of(p.proj[j], g.ids[k]);
    }
    __syncthreads();
    return n;
}

// Whether ids and ranks still give what find_groups made of them.
__device__ __forceinline__ bool still_so(const SmallParams &p, const Groups &g, const Finding &f, int groups)
{
    bool same = true;
    if (p.tokens == 1) {
        same = adapter_of(p, 0) == g.ids[0];
    } else {
#pragma unroll 1
        for (int t = threadIdx.x; t < p.tokens; t += kThreads) same = same && adapter_of(p, t) + 1 == f.bin[t];
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < groups * p.nproj; i += kThreads) {
        const int j = i / groups, k = i - j * groups;
        same = same && rank_of(p.proj[j], g.ids[k]) == g.rank[j][k];
    }
    return same;
}

// d += A B of 16 rows (tokens), 8 columns and 16 k.  A lane holds of A the rows
// lane / 4 and lane / 4 + 8, of B the column lane / 4, of d those rows and the
// columns 2 (lane % 4) and the next; of k each lane % 4 has four.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same over 32 k: `lo` and `hi` are 16 bytes of A's two rows, b of B's column.
__device__ __forceinline__ void mma32(float (&d)[4], const uint4 &lo, const uint4 &hi, const uint4 &b)
{
    mma(d, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
    mma(d, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// ldg_early_v4 of memory that the launch ahead may still have been writing when
// this one started (it is read after the wait for it): not by the read-only path.
__device__ __forceinline__ uint4 ld_early_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Units (group, kRows rows of a projection's A, slice), one after the other
__global__ void __launch_bounds__(kThreads, kShrinkCtas) small_shrink_kernel(const __grid_constant__ SmallParams p)
{
    __shared__ Groups grp;
    __shared__ union {
        alignas(16) Finding f;
        float red[2][kWarps][kGroup][kRows + 2];
    } scratch;
    auto &red = scratch.red;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kw = warp * kWarpCols + 8 * (lane & 3);
    const int t0 = lane >> 2, t1 = t0 + 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    constexpr int kSteps = kWarpCols / 32;
    const int blocks = p.row0[p.nproj];
    int groups, units;
    // the next unit from `unit` on that has something to do; its place
    int g, j, r0, slice, rank;
    auto find = [&](int unit) {
        for (; unit < units; unit += gridDim.x) {
            const int i = unit / p.slices;
            slice = unit - i * p.slices;
            g = i / blocks;
            const int row = i - g * blocks;
            j = 0;
            while (j + 1 < p.nproj && row >= p.row0[j + 1]) ++j;
            r0 = (row - p.row0[j]) * kRows;
            rank = grp.rank[j][g];
            if (r0 < rank) break;
        }
        return unit;
    };
    uint4 w[kSteps][2];
    auto load = [&]() {
        const int k0 = slice * kSlice + kw, row = r0 + t0;  // and the one 8 below
        const uint16_t *a = p.proj[j].a + ((int64_t)grp.ids[g] * p.proj[j].rank + row) * p.n_in + k0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const bool in = k0 + 32 * s < p.n_in;
            w[s][0] = in && row < rank ? ld_early_v4(a + 32 * s) : zero;
            w[s][1] = in && row + 8 < rank ? ld_early_v4(a + (int64_t)8 * p.n_in + 32 * s) : zero;
        }
    };
    // The work ahead on the stream may have let this launch start while it still
    // writes ids, ranks or the pools.  The groups are found from what is there, and
    // again after the wait for that work where ids or ranks have changed; nothing
    // else is read before it.  (100 tokens, 16 adapters of rank 32, 5120 to 2 x 17408
    // columns, passes one behind the other: 20.9 us; 21.9 with the groups found after
    // the wait, 19.4 with A read ahead of it, which would be the old A.)
    int unit;
#pragma unroll 1
    for (bool again = false;; again = true) {
        groups = find_groups(p, grp, scratch.f);
        units = groups * blocks * p.slices;
        unit = find(blockIdx.x);
        if (!again) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if (unit < units) load();
        if (again || !__syncthreads_or(!still_so(p, grp, scratch.f, groups))) break;
    }
    for (int turn = 0; unit < units; turn ^= 1) {
        const int n = grp.size[g], k0 = slice * kSlice + kw;
        const uint16_t *tok = grp.order + grp.start[g];
        const uint16_t *x0 = p.x + (int64_t)tok[t0 < n ? t0 : 0] * p.ldx + k0;
        const uint16_t *x1 = p.x + (int64_t)tok[t1 < n ? t1 : 0] * p.ldx + k0;
        uint4 lo[kSteps], hi[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const bool in = k0 + 32 * s < p.n_in;
            lo[s] = in && t0 < n ? *reinterpret_cast<const uint4 *>(x0 + 32 * s) : zero;
            hi[s] = in && t1 < n ? *reinterpret_cast<const uint4 *>(x1 + 32 * s) : zero;
        }
        float d[2][4] = {};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            mma32(d[0], lo[s], hi[s], w[s][0]);
            mma32(d[1], lo[s], hi[s], w[s][1]);
        }
        // where the partial of this thread goes: token threadIdx.x / kRows, row r0 + threadIdx.x % kRows
        const int t = threadIdx.x / kRows, r = threadIdx.x % kRows;
        float *to = t < n && r0 + r < rank
                        ? p.part[j] + ((int64_t)slice * p.tokens + tok[t]) * p.proj[j].rank + r0 + r
                        : nullptr;
        unit = find(unit + gridDim.x);
        if (unit < units) load();
        const int c = 2 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<float2 *>(&red[turn][warp][t0][8 * h + c]) = make_float2(d[h][0], d[h][1]);
            *reinterpret_cast<float2 *>(&red[turn][warp][t1][8 * h + c]) = make_float2(d[h][2], d[h][3]);
        }
        __syncthreads();  // the next unit writes the other half of `red`
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += red[turn][i][t][r];
        if (to != nullptr) *to = v;
    }
}

// Units (group, kOutputs outputs of a projection); a CTA takes a run of them, so
// that v is put together once for many units and the next unit's weights and base
// are under way while this one is added.  KS: 32 columns of B are a step, and
// `rank` has at most KS of them.
template <int KS>
__global__ void __launch_bounds__(kThreads, expand_ctas(KS)) small_expand_kernel(const __grid_constant__ SmallParams p)
{
    __shared__ Groups grp;
    // s_i v in three bf16 parts, 24 bits: nothing of the fp32 value is lost
    constexpr int kPitch = 32 * KS + 8;  // 16-byte reads of 8 rows fall into 8 different bank groups
    __shared__ union {
        alignas(16) Finding f;
        alignas(16) uint16_t vs[2][3][kGroup][kPitch];
    } scratch;
    auto &vs = scratch.vs;
    constexpr int kAtOnce = 8;  // partials a thread asks for at once
    // shrink let this launch start after its own wait: what is older is complete
    const int groups = find_groups(p, grp, scratch.f);
    if (blockIdx.x == 0)
        for (int t = threadIdx.x; t < p.tokens; t += kThreads)
            if (__ldcg(p.ids + t) >= p.count) set_status(p.status, LB_ERR_INVALID_ARGUMENT);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, q = lane & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int chunks = p.chunk0[p.nproj], units = groups * chunks;
    const int share = units / (int)gridDim.x, longer = units - share * (int)gridDim.x, cta = blockIdx.x;
    const int begin = cta * share + min(cta, longer), end = begin + share + (cta < longer ? 1 : 0);
    struct Unit {
        int g, j, out0, rank;
    };
    Unit at;
    auto find = [&](int unit) {  // the next unit with something to do
        for (; unit < end; ++unit) {
            at.g = unit / chunks;
            const int c = unit - at.g * chunks;
            at.j = 0;
            while (at.j + 1 < p.nproj && c >= p.chunk0[at.j + 1]) ++at.j;
            at.out0 = (c - p.chunk0[at.j]) * kOutputs + warp * kWarpOuts;
            at.rank = grp.rank[at.j][at.g];
            if (at.rank > 0 || p.proj[at.j].base != p.proj[at.j].y) break;
        }
        return unit;
    };
    // Column `row` of product b is output 8 (row / 2) + 2 b + row % 2 of the warp's,
    // so that a lane's columns of the four products are 8 outputs in a row, from 8 q on.
    uint4 w[KS][4], y[2];
    float scale = 1.0f;
    auto load_weights = [&]() {
        const AdapterProj &P = p.proj[at.j];
        const int id = max((int)grp.ids[at.g], 0);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int o = at.out0 + 8 * (row >> 1) + 2 * b + (row & 1);
            const uint16_t *B = P.b + ((int64_t)id * P.n_out + o) * P.rank + 8 * q;
#pragma unroll
            for (int k = 0; k < KS; ++k) w[k][b] = o < P.n_out && 32 * k + 8 * q < at.rank ? ldg_early_v4(B + 32 * k) : zero;
        }
        scale = P.scale != nullptr ? __ldg(P.scale + id) : 1.0f;
    };
    auto load_base = [&]() {
        const AdapterProj &P = p.proj[at.j];
        const int o = at.out0 + 8 * q;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            y[h] = o < P.n_out && row + 8 * h < grp.size[at.g]
                       ? *reinterpret_cast<const uint4 *>(P.base + (int64_t)grp.order[grp.start[at.g] + row + 8 * h] * P.ldbase + o)
                       : zero;
    };
    int unit = find(begin);
    if (unit < end) load_weights();
    pdl_wait();
    pdl_launch_dependents();
    if (unit < end) load_base();
    int turn = 0, vg = -1, vj = -1;  // whose v is in vs[turn]
    while (unit < end) {
        const Unit u = at;
        const AdapterProj &P = p.proj[u.j];
        const int n = grp.size[u.g], o = u.out0 + 8 * q;
        const uint16_t *tok = grp.order + grp.start[u.g];
        if (u.rank > 0 && (u.g != vg || u.j != vj)) {
            turn ^= 1;  // some threads may still read the other half
            vg = u.g;
            vj = u.j;
            const int64_t next = (int64_t)p.tokens * P.rank;
            for (int i = threadIdx.x; i < n * 16 * KS; i += kThreads) {
                const int t = i / (16 * KS), r = i % (16 * KS) * 2;  // and r + 1
                float2 v = make_float2(0.0f, 0.0f);
                if (r < u.rank) {
                    const float *part = p.part[u.j] + (int64_t)tok[t] * P.rank + r;
                    for (int s0 = 0; s0 < p.slices; s0 += kAtOnce) {
                        float2 e[kAtOnce];
#pragma unroll
                        for (int s = 0; s < kAtOnce; ++s)
                            e[s] = s0 + s < p.slices ? *reinterpret_cast<const float2 *>(part + (s0 + s) * next) : make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int s = 0; s < kAtOnce; ++s) v.x += e[s].x, v.y += e[s].y;
                    }
                }
                v.x *= scale;
                v.y = r + 1 < u.rank ? v.y * scale : 0.0f;  // nothing was written past the rank
#pragma unroll
                for (int k = 0; k < 3; ++k) {  // truncated, so that no part can overflow
                    const uint32_t x = __float_as_uint(v.x) & 0xffff0000u, z = __float_as_uint(v.y) & 0xffff0000u;
                    *reinterpret_cast<uint32_t *>(&vs[turn][k][t][r]) = x >> 16 | z;
                    v.x = isfinite(v.x) ? v.x - __uint_as_float(x) : 0.0f;
                    v.y = isfinite(v.y) ? v.y - __uint_as_float(z) : 0.0f;
                }
            }
            __syncthreads();
        }
        float d[4][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            if (32 * k < u.rank) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const uint4 lo = row < n ? *reinterpret_cast<const uint4 *>(&vs[turn][i][row][32 * k + 8 * q]) : zero;
                    const uint4 hi = row + 8 < n ? *reinterpret_cast<const uint4 *>(&vs[turn][i][row + 8][32 * k + 8 * q]) : zero;
#pragma unroll
                    for (int b = 0; b < 4; ++b) mma32(d[b], lo, hi, w[k][b]);
                }
            }
        }
        unit = find(unit + 1);
        if (unit < end) load_weights();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (u.rank > 0) {
                uint32_t e[4] = {y[h].x, y[h].y, y[h].z, y[h].w};
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    e[b] = pack_bf162(__uint_as_float(e[b] << 16) + d[b][2 * h], __uint_as_float(e[b] & 0xffff0000u) + d[b][2 * h + 1]);
                y[h] = make_uint4(e[0], e[1], e[2], e[3]);
            }
            if (o < P.n_out && row + 8 * h < n)
                *reinterpret_cast<uint4 *>(P.y + (int64_t)tok[row + 8 * h] * P.ldy + o) = y[h];
        }
        if (unit < end) load_base();
    }
}

int small_slices(int n_in) { return (n_in + kSlice - 1) / kSlice; }

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
    p.slices = small_slices(a.n_in);
    p.status = dev.status;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    int rank = 0;
    for (int j = 0; j < a.nproj; ++j) {
        p.proj[j] = a.proj[j];
        p.part[j] = reinterpret_cast<float *>(ws);
        ws += align256(sizeof(float) * (size_t)p.slices * (size_t)M * (size_t)a.proj[j].rank);
        p.chunk0[j + 1] = p.chunk0[j] + (a.proj[j].n_out + kOutputs - 1) / kOutputs;
        p.row0[j + 1] = p.row0[j] + (a.proj[j].rank + kRows - 1) / kRows;
        rank = std::max(rank, a.proj[j].rank);
    }
    // groups: one for each adapter in use and for the tokens without one, and the full ones
    const int groups = std::min(M, std::min(a.count + 1, M) + M / kGroup);
    const int sms = dev.sm_count;
    auto grid = [&](int units, int ctas) { return dim3((unsigned)std::min(units, sms * ctas)); };
    const cudaError_t e = launch_pdl(small_shrink_kernel, grid(groups * p.row0[a.nproj] * p.slices, kShrinkCtas), p, stream);
    if (e != cudaSuccess) return e;
    const int units = groups * p.chunk0[a.nproj];
    return rank <= 32   ? launch_pdl(small_expand_kernel<1>, grid(units, expand_ctas(1)), p, stream)
           : rank <= 64 ? launch_pdl(small_expand_kernel<2>, grid(units, expand_ctas(2)), p, stream)
                        : launch_pdl(small_expand_kernel<4>, grid(units, expand_ctas(4)), p, stream);
}

size_t small_workspace(int M, int n_in, int nproj, const int *ranks)
{
    size_t b = 0;
    for (int j = 0; j < nproj; ++j)
        b += align256(sizeof(float) * (size_t)small_slices(n_in) * (size_t)M * (size_t)ranks[j]);
    return b;
}

}  // namespace

// The most tokens of a call that runs here: see the top of this file.
static int most_small_tokens(int count)
{
    return std::max(std::min(512, 128 + 48 * count), std::min(kAdapterSmallTokens, 24 * count));
}
static bool small_batch(int tokens, int count) { return tokens <= most_small_tokens(count); }

// Enough for every smaller number of tokens too: the partial sums of a small batch,
// which grow with n_in, can be more than a larger one's plan and tiles.
size_t adapters_workspace_bytes(int tokens, int n_in, int count, int nproj, const int *ranks)
{
    const size_t small = small_workspace(std::min(tokens, most_small_tokens(count)), n_in, nproj, ranks);
    return small_batch(tokens, count) ? small : std::max(small, adapters_mma_workspace_bytes(tokens, count, nproj, ranks));
}

cudaError_t adapters_prepare_device(const DeviceInfo &dev) { return adapters_mma_prepare_device(dev); }

cudaError_t adapters_forward(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    return small_batch(a.tokens, a.count) ? small_adapters(a, dev, stream) : adapters_mma_forward(a, dev, stream);
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
