// lb_adapters_mma.cu - low-rank adapters of many requests on the tensor
// cores: batches past a few tokens, and the backward pass.
//
//     v = s_i A_i x,  y = base + B_i v                        (forward)
//     u = s_i B_i^T dy,  dx = dx_base + A_i^T u,
//     dA_i = sum u x^T,  dB_i = sum dy v^T                    (backward)
//
// With r <= 128 against thousands of columns, every product streams one wide
// operand (x, dy, base and y) past a thin one, so DRAM bounds them; the tensor
// cores only have to keep out of the way.  What the layout settles is that
// each wide operand crosses once a product whatever order the tokens come in:
//
//   plan    one CTA sorts the tokens by adapter (a stable counting sort) into
//           tiles of 128 slots, each of one adapter; a slot past an adapter's
//           tokens holds the row number `tokens`, which no tensor has: TMA
//           reads zeros there
//   shrink  a tile's rows of x against A_i (or of dy against B_i), every CTA an
//           equal share of all the tiles' K-blocks; the rows come by TMA; v is
//           kept as a sum of bf16 (what a first one leaves goes to a second,
//           and what that leaves to a third)
//   expand  v against B_i (or A_i), 128 x 128 outputs at a time; base comes by
//           TMA ahead of use, the sum goes back to its row
//   wgrad   x^T u and dy^T v over an adapter's slots, both operands MN-major
//           as they lie, every CTA an equal share again
//   finish  after shrink and wgrad: the products that fell to several CTAs,
//           their fp32 sums added in the CTAs' order
//
// Two choices keep fp32 results fp32.  The tensor cores take bf16, so expand
// multiplies the first two parts of v (2^-16 of v is lost, under a bf16 output
// step of 2^-8) and wgrad all three (24 bits, nothing lost).  And they truncate
// as they accumulate, about 2^-26 of the sum a step, all to one side: 1.6e-5
// of v over 16384 columns.  So no sum stays in tensor memory for more than
// kSegment K-blocks; the epilogue warps add those sums up in registers, rounding
// to nearest.  The extra products and reads hide behind the wide operand.
//
// A launch begins as soon as the one before allows and waits only for what that
// one writes.  plan reads nothing ahead of its wait; of the kernels behind it each
// reads the plan, the weights and the wide operand before its wait, which are
// older: each of them, and plan, lets the next begin only after its own wait, so
// that all launches but the last one are complete, whatever came before plan.  In
// the backward pass wgrad goes before expand, and expand, which needs nothing of
// it, begins on the SMs that wgrad leaves.  Measured on the device, passes one
// behind the other, 8192 tokens of 5120 columns, 8 adapters of rank 64: forward to
// 5120 columns 67 us (of it shrink 23, 3.7 TB/s; finish 3; expand 30, 5.6 TB/s over
// the base read and y written; 63 with plan's counting ahead of its wait), backward
// from 17408 columns, 4 adapters, 198 us (shrink 72 us, 5.1 TB/s; wgrad 74, 5.0
// TB/s; expand 30; finish 3 and 10).  333 tokens, 3 adapters of rank 8, 4096 x 4096,
// backward 26 us: six launches of 3 to 6 us, each a chain of reads that depend on one
// another.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_operators.h"
#include "lb_tc.cuh"

namespace lb {
namespace {

using namespace tc;

constexpr int TM = 128;               // slots of a tile
constexpr uint32_t kBox = 64 * 128;   // 64 rows (or slots) of 64 two-byte elements
constexpr int kSegment = 4;           // K-blocks that are summed in tensor memory
constexpr int kParts = 3;             // bf16 that v is the sum of

// ------------------------------------------------------------ the plan
struct alignas(16) Tile {
    int adapter;      // -1: tokens without an adapter
    int rows;         // slots in use, from 1 to TM
    int first, last;  // the first and last of its tokens, which are in order
    __device__ __forceinline__ bool run() const { return last - first == rows - 1; }  // none missing between
};
struct Plan {
    int *counts;   // tiles, those of adapters (the first ones), 64-slot blocks of adapters
    Tile *tiles;
    int *perm;     // [tiles][TM]: the token of each slot, `tokens` for none
    int *block0;   // [count + 1]: blocks of the adapters before; each has ceil(its tokens / 64)
    int *tile0;    // [count]: tiles of the adapters before
};

struct PlanParams {
    const int32_t *ids;
    int tokens, count;
    Plan plan;
    int *status;
};

constexpr int kPlanThreads = 1024, kPlanWarps = 32;
constexpr int kHeld = 8192;  // tokens that stay in shared memory between the two passes
constexpr int kBinBits = 11;
static_assert(LB_MAX_ADAPTERS < 1 << kBinBits, "a bin, and above it a place");
constexpr int kPlanTokens = 1 << 20;  // the most; the sums over adapters of tiles and blocks share 32 bits
static_assert(kPlanTokens / TM + LB_MAX_ADAPTERS < 1 << 14 && kPlanTokens / 64 + LB_MAX_ADAPTERS < 1 << 18, "tiles, blocks");

// Each warp takes a run of tokens in order, so that an adapter's tokens keep
// their order and sums over them do not depend on timing.  One CTA runs this
// once, so its instructions come from far away: the code is kept short (loops
// stay rolled; unrolled it took twice as long).  The ids may have been written by
// the work ahead on the stream, so they are read after the wait for it.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p)
{
    extern __shared__ int hist[];  // [warp][bin]; bin `count`: no adapter
    __shared__ uint32_t sums[kPlanWarps];
    __shared__ int first_tile[LB_MAX_ADAPTERS + 1], total[LB_MAX_ADAPTERS + 1];
    __shared__ int held[kHeld];  // bins, with places among a warp's tokens of a bin
    const int bins = p.count + 1, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int rounds = (p.tokens + kPlanThreads - 1) / kPlanThreads;
    const int t0 = w * rounds * 32 + lane;
    int *mine = hist + w * bins;
    const bool hold = p.tokens <= kHeld;
    auto bin_of = [&](int id) {
        if (id >= p.count) set_status(p.status, LB_ERR_INVALID_ARGUMENT);
        return id < 0 || id >= p.count ? p.count : id;
    };
#pragma unroll 1
    for (int i = tid; i < kPlanWarps * bins; i += kPlanThreads) hist[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    if (hold) {
        int ids[kHeld / kPlanThreads];
#pragma unroll
        for (int i = 0; i < kHeld / kPlanThreads; ++i) {
            const int t = i * kPlanThreads + tid;
            ids[i] = t < p.tokens ? __ldcg(p.ids + t) : -1;
        }
#pragma unroll
        for (int i = 0; i < kHeld / kPlanThreads; ++i) held[i * kPlanThreads + tid] = bin_of(ids[i]);
    }
    __syncthreads();
    auto put = [&](int t, int slot, bool first, bool last) {
        p.plan.perm[slot] = t;
        if (first) p.plan.tiles[slot / TM].first = t;
        if (last) p.plan.tiles[slot / TM].last = t;
    };
    int all_tiles = 0, tile0 = 0, block0 = 0, all_blocks = 0;
    // pass 0 counts each warp's tokens of each bin, pass 1 gives them their slots:
    // from the places that pass 0 kept, or by counting again
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int i = 0; i < rounds; ++i) {
            const int t = t0 + 32 * i;
            int b = -1;
            if (t < p.tokens) b = hold ? held[t] : bin_of(__ldcg(p.ids + t));
            const uint32_t same = __match_any_sync(0xffffffffu, b);  // the lanes with the same bin
            const int had = b >= 0 ? mine[b] : 0;
            __syncwarp();
            if (b >= 0) {
                const int rank = __popc(same & ((1u << lane) - 1u));
                const int at = had + rank;
                if (pass == 1)
                    put(t, first_tile[b] * TM + at, at % TM == 0, at % TM == TM - 1 || at == total[b] - 1);
                else if (hold)
                    held[t] = b | at << kBinBits;  // its place among the warp's
                if (rank == 0) mine[b] = had + __popc(same);
            }
            __syncwarp();
        }
        if (pass == 1) break;
        __syncthreads();
        // per bin: its tokens, and where each warp's share of them begins
#pragma unroll 1
        for (int b = w; b < bins; b += kPlanWarps) {
            const int k = hist[lane * bins + b];
            int inc = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            hist[lane * bins + b] = inc - k;
            if (lane == 31) total[b] = inc;
        }
        __syncthreads();
        // one sum over the adapters of two counts: tiles, and above them blocks
        const int n = tid < p.count ? total[tid] : 0;
        const int tiles = (n + TM - 1) / TM;
        constexpr int kTileBits = 14;
        const uint32_t v = (uint32_t)tiles | (uint32_t)((n + 63) / 64) << kTileBits;
        uint32_t inc = v;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sums[w] = inc;
        __syncthreads();
        uint32_t all = sums[lane];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, all, o);
            if (lane >= o) all += u;
        }
        const uint32_t below = __shfl_sync(0xffffffffu, all, max(w - 1, 0));
        all = __shfl_sync(0xffffffffu, all, 31);
        const uint32_t before = inc - v + (w > 0 ? below : 0);
        all_tiles = (int)(all & ((1u << kTileBits) - 1));
        tile0 = (int)(before & ((1u << kTileBits) - 1));
        all_blocks = (int)(all >> kTileBits);
        block0 = (int)(before >> kTileBits);
        if (tid < p.count) first_tile[tid] = tile0;
        if (tid == 0) first_tile[p.count] = all_tiles;
        __syncthreads();
        if (hold) break;
    }
    if (hold) {
#pragma unroll 2
        for (int i = 0; i < rounds; ++i) {
            const int t = t0 + 32 * i;
            if (t >= p.tokens) break;
            const int v = held[t], b = v & ((1 << kBinBits) - 1);
            const int at = mine[b] + (v >> kBinBits);
            put(t, first_tile[b] * TM + at, at % TM == 0, at % TM == TM - 1 || at == total[b] - 1);
        }
    }
    if (tid < p.count) {
        p.plan.tile0[tid] = tile0;
        p.plan.block0[tid] = block0;
    }
    if (tid == 0) {
        p.plan.counts[0] = all_tiles + (total[p.count] + TM - 1) / TM;
        p.plan.counts[1] = all_tiles;
        p.plan.counts[2] = p.plan.block0[p.count] = all_blocks;
    }
#pragma unroll 1
    for (int b = w; b < bins; b += kPlanWarps) {  // the bin's tiles, and its slots without a token
        const int m = total[b], at = first_tile[b], end = (m + TM - 1) / TM * TM;
#pragma unroll 1
        for (int i = lane; i * TM < m; i += 32) {
            p.plan.tiles[at + i].adapter = b < p.count ? b : -1;
            p.plan.tiles[at + i].rows = min(TM, m - i * TM);
        }
#pragma unroll 1
        for (int s = m + lane; s < end; s += 32) p.plan.perm[at * TM + s] = p.tokens;
    }
}

// ------------------------------------------------------------ loads
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// True in one thread of a converged warp.  The loops that issue MMAs and copies
// run under it rather than under `lane == 0`: what those instructions take must
// be uniform, which the compiler then knows (an MMA of 128 x 64 x 16 issued
// under a lane test took 110 cycles).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// An MMA by the low words of its operands' descriptors, which hold the address
// in 16-byte units; the high words are the same for every K- or MN-major tile.
constexpr uint32_t kDescHigh = 64u | (1u << 14) | (2u << 29);
__device__ __forceinline__ void umma_lo(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(tmem_d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
        : "memory");
}
// MN-major operand with 128-byte swizzle: 64-wide MN chunks kBox bytes apart,
// 8-row K groups 1024 bytes apart; 16 rows of K are 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(kBox >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// bf16 operands, fp32 accumulation, M = 128; A and B MN-major where asked.
__device__ __forceinline__ uint32_t idesc_of(int n, bool a_mn, bool b_mn)
{
    return instr_desc(1, TM, n) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16);
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4 &v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Two bf16 and two fp32 values added, back in bf16.
__device__ __forceinline__ uint32_t add_bf162(uint32_t b, uint32_t lo, uint32_t hi)
{
    return pack_bf162(__uint_as_float(b << 16) + __uint_as_float(lo), __uint_as_float(b & 0xffff0000u) + __uint_as_float(hi));
}

// Where a wait gave up, copies may still be in flight to this CTA's shared
// memory, and which ones is not kept; they land within microseconds.
__device__ __forceinline__ void drain_copies()
{
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
}

// How a tile's rows come.  Consecutive ones, as a prompt's tokens are, in one
// TMA box.  TMA's gather of four rows takes the time of a far larger box (84 MB
// of x took 37 us so, 25 us in boxes; a single tile with a break in it held the
// backward pass at 8192 tokens for 30 us), so the rows of other tiles come as
// 16-byte copies of the threads of kLoaders warps.  A stage's full barrier
// counts kFull arrivals: of those threads as their copies land, and of the one
// that announces the TMA bytes, which arrives for all where TMA brings the rows.
// (A writer's own wait and proxy fence before its arrival made a K-block of such
// a tile wait for every copy under way; the reader of the stage has the fence.)
struct Rows {
    CUtensorMap box;  // a tile's rows (of a K-block for wgrad) x 64 columns
    const uint16_t *p;
    int64_t ld;
    int cols;
};
constexpr int kLoaders = 4;
constexpr int kLoadThreads = 32 * kLoaders;
__device__ __forceinline__ void loaders_meet() { asm volatile("bar.sync 2, %0;" ::"n"(kLoadThreads) : "memory"); }
constexpr int kFull = 1 + kLoadThreads;
__device__ __forceinline__ void mbar_arrive_for_loaders(uint32_t bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "n"(kLoadThreads)
                 : "memory");
}
// Arrives when this thread's copies so far have landed.
__device__ __forceinline__ void mbar_arrive_after_copies(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 bytes to shared memory, zeros where `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// This thread's part of ROWS rows x 64 columns: every kStep-th row from tid / 8
// on, 16 bytes at chunk tid % 8, in the layout of a TMA box.  The rows' addresses
// are found once, so that a copy is an addition and the copy itself: with a
// multiplication in each, four warps could not keep up with a weight gradient
// (the backward pass of 8192 tokens in any order, 276 us; 236 us so).  Rows that are not `there` are not read
// (`strict`: zeros).
template <int ROWS>
struct Copier {
    static constexpr int kStep = kLoadThreads / 8, kN = ROWS / kStep;
    const uint16_t *src[kN];
    uint32_t there;
    int r0, chunk;
    template <typename F>
    __device__ __forceinline__ void set(const uint16_t *p, int64_t ld, int used, int tid, F row)
    {
        r0 = tid >> 3;
        chunk = tid & 7;
        there = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int r = r0 + kStep * i;
            src[i] = p;
            if (r < used) {
                src[i] = p + row(r) * ld;
                there |= 1u << i;
            }
        }
    }
    __device__ __forceinline__ void rows(const uint16_t *p, int64_t ld, const int *perm, int used, int tid)
    {
        set(p, ld, used, tid, [&](int r) { return perm[r]; });
    }
    __device__ __forceinline__ void run(const uint16_t *p, int64_t ld, int first, int used, int tid)
    {
        set(p, ld, used, tid, [&](int r) { return first + r; });
    }
    // BOXES of 64 columns from `col` on
    template <int BOXES>
    __device__ __forceinline__ void copy(uint32_t dst, uint32_t box, int cols, int col, bool strict) const
    {
        const int c = col + 8 * chunk;
        const uint32_t at = dst + r0 * 128u + (uint32_t)((chunk ^ (r0 & 7)) << 4);  // rows kStep apart: the same swizzle
        if (c + 64 * (BOXES - 1) < cols) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const bool in = there >> i & 1u;
                const uint16_t *from = src[i] + c;
#pragma unroll
                for (int b = 0; b < BOXES; ++b)
                    if (strict || in) copy16(at + 128u * kStep * i + b * box, from + 64 * b, in);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
#pragma unroll
                for (int b = 0; b < BOXES; ++b) {
                    const bool in = (there >> i & 1u) && c + 64 * b < cols;
                    copy16(at + 128u * kStep * i + b * box, src[i] + (in ? c + 64 * b : 0), in);
                }
            }
        }
    }
};

__device__ __forceinline__ int used_rank(const int32_t *ranks, int rank, int adapter)
{
    return ranks == nullptr ? rank : max(0, min(rank, __ldg(ranks + adapter)));
}

// `work` K-blocks in equal runs over up to `most` CTAs, at least `least` to
// each: CTA c has start(c) .. start(c + 1) - 1.
// Shrink takes 4 or more: sums that a CTA shares cost a read and a write of them.
// A weight gradient has few K-blocks where there are few tokens, and one each
// spreads its products: at 4 instead of 1, 30 tokens of 2 adapters took 8 us more,
// 148 tokens of 4 adapters of rank 64 10 us more.
constexpr int kLeastBlocks = 4;
struct Shares {
    int ctas, base, rem;
    __device__ __forceinline__ Shares(int work, int most, int least)
    {
        ctas = max(1, min(most, work / least));
        base = work / ctas;
        rem = work - base * ctas;
    }
    __device__ __forceinline__ int start(int c) const { return c * base + min(c, rem); }
    __device__ __forceinline__ int owner(int w) const
    {
        const int longer = rem * (base + 1);
        return w < longer ? w / (base + 1) : rem + (w - longer) / base;
    }
    // A CTA's sums of a product that it shares: its first product's are slot 0
    // of its two, its last one's slot 1.
    __device__ __forceinline__ int slot(int c, int product_begin) const { return 2 * c + (start(c) < product_begin); }
};

// ------------------------------------------------------------ shrink
// v = s_i W_i x of every tile's rows, W_i [rank x K] (K-major: A_i) or [K x rank]
// (MN-major: B_i).  Persistent CTAs with equal shares of all K-blocks of all
// jobs and tiles, in order.  Splitting each product over a cluster of 2, 4 or 8
// CTAs instead left a third of the SMs idle at the end of the backward pass
// (104 us at 8192 tokens, 5120 and 17408 columns), and letting the last CTA of
// a product add the others' sums held 13 thousand cycles behind the last MMA.
struct ShrinkJob {
    Rows x;
    CUtensorMap w;
    int nkb, rank, mn;  // K-blocks of 64 columns
    const int32_t *ranks;
    const float *scale;
    uint16_t *v[kParts];  // [slots][rank] each; the third may be null
};
struct ShrinkParams {
    ShrinkJob job[kMaxSiblings];
    int njobs, per_tile;  // K-blocks of a tile in all jobs
    Plan plan;
    float *part;  // [slot][TM][part_rank]: sums of products that several CTAs share
    int part_rank, ctas;
    int *status;
};

constexpr int kShrinkThreads = 32 * (2 + 4 + kLoaders - 1);
constexpr uint32_t kXBytes = TM * 128;  // a K-block of a tile's rows: 64 columns
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
template <int NK>
struct Shrink {
    static constexpr uint32_t kStage = kXBytes + NK * kBox;
    static constexpr int kStages = NK == 1 ? 8 : 6;
    static constexpr size_t kSmem = 1024 + kStages * kStage + 256;
};

// Four elements of v from their sums: scaled, zero past the adapter's rank, and
// split into bf16 parts, each what the ones before leave (exactly; an infinity
// or NaN is all in the first, and a finite value that would round to one leaves
// the largest bf16 there).
__device__ __forceinline__ void store_v(const ShrinkJob &J, int64_t at, int c, int rank, float scale, const float4 &s)
{
    float f[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = c + e < rank ? f[e] * scale : 0.0f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
        if (J.v[k] == nullptr) break;
        float g[4] = {f[0], f[1], f[2], f[3]};
        if (k == 0) {
            const float most = __int_as_float(0x7f7f0000);  // of bf16
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (fabsf(g[e]) < __int_as_float(0x7f800000)) g[e] = fminf(fmaxf(g[e], -most), most);
        }
        const uint2 o = make_uint2(pack_bf162(g[0], g[1]), pack_bf162(g[2], g[3]));
        *reinterpret_cast<uint2 *>(J.v[k] + at) = o;
        const float h[4] = {__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xffff0000u), __uint_as_float(o.y << 16),
                            __uint_as_float(o.y & 0xffff0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = fabsf(h[e]) < __int_as_float(0x7f800000) ? f[e] - h[e] : 0.0f;
    }
}

template <int NK>
__global__ void __launch_bounds__(kShrinkThreads, 1) shrink_kernel(const __grid_constant__ ShrinkParams p)
{
    using S = Shrink<NK>;
    constexpr int kRank = 64 * NK;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + S::kStages * S::kStage;
    const uint32_t full0 = bars, empty0 = full0 + 8 * S::kStages, accf0 = empty0 + 8 * S::kStages, acce0 = accf0 + 16;
    const uint32_t drain = acce0 + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (drain + 8 - raw));
    __shared__ int abort_shared;
    volatile int &abort_flag = abort_shared;

    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < S::kStages; ++s) {
                mbar_init(full0 + 8 * s, kFull);
                mbar_init(empty0 + 8 * s, 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(accf0 + 8 * b, 1);
                mbar_init(acce0 + 8 * b, 4);
            }
            mbar_init(drain, 1);
            abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 256);
        tc_fence_before();
    } else if (warp == 0 && elect_one()) {
        for (int j = 0; j < p.njobs; ++j) {
            prefetch_map(&p.job[j].x.box);
            prefetch_map(&p.job[j].w);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int live = p.plan.counts[1], cta = blockIdx.x;
    const Shares shares(live * p.per_tile, p.ctas, kLeastBlocks);
    const int w0 = cta < shares.ctas ? shares.start(cta) : 0, w1 = cta < shares.ctas ? shares.start(cta + 1) : 0;
    // the part of one product that begins at K-block w of this CTA's share
    struct Piece {
        int tile, job, kb, n;
    };
    auto piece_at = [&](int w) {
        Piece q;
        q.job = 0;
        int nkb = p.job[0].nkb;
        while (w >= nkb * live) {
            w -= nkb * live;
            nkb = p.job[++q.job].nkb;
        }
        q.tile = w / nkb;
        q.kb = w - q.tile * nkb;
        return q;
    };
    auto piece = [&](int w) {
        Piece q = piece_at(w);
        q.n = min(p.job[q.job].nkb - q.kb, w1 - w);
        return q;
    };
    // (What the K-block loops below need is in registers before they start: a
    // parameter read there costs as much as an MMA.)

    const int loader = warp == 0 ? 0 : warp - 5;  // warps 0 and 6 ..
    if (warp == 0 || warp > 5) {
        int g = 0;  // K-blocks of the pieces so far
        for (int w = w0; w < w1;) {  // to the end in every loader, whatever happens: they meet
            const Piece q = piece(w);
            const ShrinkJob &J = p.job[q.job];
            const Tile T = p.plan.tiles[q.tile];
            // rows past the tile's may be anything: they end in rows of v that are zeros
            const bool run = T.run(), mn = J.mn != 0, two = mn && J.rank > 64;
            const uint32_t w_bytes = two ? 2 * kBox : mn ? kBox : (uint32_t)((J.rank + 15) & ~15) * 128u;
            const CUtensorMap *mx = &J.x.box, *mw = &J.w;
            int s = g % S::kStages;
            uint32_t ph = ((uint32_t)(g / S::kStages) & 1u) ^ 1u;
            auto load_w = [&](int kb) {
                const uint32_t sw = base + s * S::kStage + kXBytes, bar = full0 + 8 * s;
                tma_load_3d(sw, mw, mn ? 0 : 64 * kb, mn ? 64 * kb : 0, T.adapter, bar);
                if (two) tma_load_3d(sw + kBox, mw, 64, 64 * kb, T.adapter, bar);
            };
            if (run && loader == 0) {
                if (elect_one()) {
                    for (int kb = q.kb; kb < q.kb + q.n; ++kb) {
                        if (!mbar_wait(empty0 + 8 * s, ph) || abort_flag) {
                            abort_flag = 1;
                            break;
                        }
                        mbar_arrive_expect_tx(full0 + 8 * s, kXBytes + w_bytes);
                        mbar_arrive_for_loaders(full0 + 8 * s);
                        load_w(kb);
                        tma_load_2d(base + s * S::kStage, mx, 64 * kb, T.first, full0 + 8 * s);
                        if (++s == S::kStages) s = 0, ph ^= 1;
                    }
                }
                __syncwarp();
            } else if (!run) {
                const uint16_t *x = J.x.p;
                const int64_t ld = J.x.ld;
                const int cols = J.x.cols;
                Copier<TM> mine;
                mine.rows(x, ld, p.plan.perm + q.tile * TM, T.rows, 32 * loader + lane);
                loaders_meet();  // the first is here, so nobody is ahead of the ring
                for (int kb = q.kb; kb < q.kb + q.n; ++kb) {
                    const bool ok = !abort_flag && mbar_wait(empty0 + 8 * s, ph);
                    if (!__all_sync(0xffffffffu, ok)) {
                        abort_flag = 1;
                        break;
                    }
                    if (loader == 0 && elect_one()) {
                        mbar_arrive_expect_tx(full0 + 8 * s, w_bytes);
                        load_w(kb);
                    }
                    __syncwarp();
                    mine.copy<1>(base + s * S::kStage, 0, cols, 64 * kb, false);
                    mbar_arrive_after_copies(full0 + 8 * s);
                    if (++s == S::kStages) s = 0, ph ^= 1;
                }
            }
            g += q.n;
            w += q.n;
        }
        // after an abort: copies in flight land within microseconds
        if (abort_flag) drain_copies();
    } else if (warp == 1) {
        if (elect_one()) {
            int s = 0, na = 0;
            uint32_t ph = 0;
            for (int w = w0; w < w1 && !abort_flag;) {
                const Piece q = piece(w);
                const ShrinkJob &J = p.job[q.job];
                const bool mn = J.mn != 0;
                const uint32_t idesc = idesc_of((J.rank + 15) & ~15, false, mn);
                const uint32_t a0 = (uint32_t)smem_desc(base);
                const uint32_t b0 = mn ? (uint32_t)smem_desc_mn(base + kXBytes) : (uint32_t)smem_desc(base + kXBytes);
                const uint32_t bstep = mn ? 2048u >> 4 : 32u >> 4;
                const bool copied = !p.plan.tiles[q.tile].run();
                for (int i = 0; i < q.n; ++i) {
                    const int b = na & 1;
                    const bool first = i % kSegment == 0;
                    if ((first && !mbar_wait(acce0 + 8 * b, ((uint32_t)(na >> 1) & 1u) ^ 1u)) ||
                        !mbar_wait(full0 + 8 * s, ph) || abort_flag) {
                        abort_flag = 1;
                        break;
                    }
                    if (copied) fence_async_shared();  // the loaders' writes, before the MMA reads them
                    tc_fence_after();
                    const uint32_t at = (uint32_t)s * (S::kStage >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_lo(tmem + 128 * b, a0 + at + 2 * kk, b0 + at + bstep * kk, idesc, !first || kk != 0 ? 1u : 0u);
                    umma_commit(empty0 + 8 * s);
                    if (i % kSegment == kSegment - 1 || i + 1 == q.n) {
                        umma_commit(accf0 + 8 * b);
                        ++na;
                    }
                    if (++s == S::kStages) s = 0, ph ^= 1;
                }
                w += q.n;
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else {
        // a row a lane: the segments' sums in registers
        const int quad = warp & 3, row = 32 * quad + lane;
        int na = 0;
        for (int w = w0; w < w1;) {
            const Piece q = piece(w);
            const ShrinkJob &J = p.job[q.job];
            const int nr = (J.rank + 15) & ~15;
            float sum[kRank];
#pragma unroll
            for (int c = 0; c < kRank; ++c) sum[c] = 0.0f;
            bool ok = true;
            for (int i = 0; i < q.n; i += kSegment, ++na) {
                const int b = na & 1;
                ok = !abort_flag && mbar_wait(accf0 + 8 * b, (uint32_t)(na >> 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kRank; c += 16) {
                    if (c < nr) {
                        uint32_t v[16];
                        tmem_ld16(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * b + c), v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[c + e] += __uint_as_float(v[e]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * b);
            }
            if (!ok) {
                abort_flag = 1;
                break;
            }
            w += q.n;
            const Tile T = p.plan.tiles[q.tile];
            if (q.n < J.nkb) {  // the rest is with this CTA's neighbours: their sums meet in shrink_finish_kernel
                float *mine = p.part + ((int64_t)shares.slot(cta, w - q.n - q.kb) * TM + row) * p.part_rank;
#pragma unroll
                for (int c = 0; c < kRank; c += 4)
                    if (c < J.rank) *reinterpret_cast<float4 *>(mine + c) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
                continue;
            }
            const int rank = row < T.rows ? used_rank(J.ranks, J.rank, T.adapter) : 0;
            const float scale = J.scale != nullptr ? __ldg(J.scale + T.adapter) : 1.0f;
            const int64_t at = ((int64_t)q.tile * TM + row) * J.rank;
#pragma unroll
            for (int c = 0; c < kRank; c += 4)
                if (c < J.rank) store_v(J, at + c, c, rank, scale, make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) set_status(p.status, LB_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// The products of shrink that several CTAs share, kFinishRows rows a unit.
constexpr int kFinishThreads = 256, kFinishRows = 16;
// Sums a thread asks for at once: a long row in a small batch is shared by many
// CTAs (40 tokens, 16160 columns: 60 of them, 10 us in fours).
constexpr int kAtOnce = 16;
__global__ void __launch_bounds__(kFinishThreads) shrink_finish_kernel(const __grid_constant__ ShrinkParams p)
{
    // one thread finds what a unit adds: the index arithmetic of all threads
    // took longer than the sums
    struct Found {
        int tile, job, used, rows, more;  // more: shared sums after the first
        float scale;
        const float *first, *rest;
    };
    __shared__ Found found;
    // the plan was complete before shrink let this launch start
    const int live = p.plan.counts[1], units = live * p.njobs * (TM / kFinishRows);
    auto find = [&](int u) {
        if (threadIdx.x == 0 && u < units) {
            const Shares shares(live * p.per_tile, p.ctas, kLeastBlocks);
            const int product = u / (TM / kFinishRows), tile = product % live, job = product / live;
            const ShrinkJob &J = p.job[job];
            int begin = tile * J.nkb;
            for (int j = 0; j < job; ++j) begin += p.job[j].nkb * live;
            const int first = shares.owner(begin), last = shares.owner(begin + J.nkb - 1);
            found.more = last - first;
            if (last > first) {
                const Tile T = p.plan.tiles[tile];
                found.tile = tile;
                found.job = job;
                found.rows = T.rows;
                found.used = used_rank(J.ranks, J.rank, T.adapter);
                found.scale = J.scale != nullptr ? __ldg(J.scale + T.adapter) : 1.0f;
                // the others begin their shares inside the product
                found.first = p.part + (int64_t)shares.slot(first, begin) * TM * p.part_rank;
                found.rest = p.part + (int64_t)2 * (first + 1) * TM * p.part_rank;
            }
        }
    };
    find(blockIdx.x);
    pdl_wait();
    pdl_launch_dependents();
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        __syncthreads();
        const Found f = found;
        __syncthreads();
        find(u + gridDim.x);
        if (f.more == 0) continue;
        const ShrinkJob &J = p.job[f.job];
        const int cols = J.rank / 4, stride = 2 * TM * p.part_rank;
        for (int i = threadIdx.x; i < kFinishRows * cols; i += kFinishThreads) {
            const int r = i / cols, row = u % (TM / kFinishRows) * kFinishRows + r, c = 4 * (i - r * cols);
            const int at = row * p.part_rank + c;
            float4 s = __ldcg(reinterpret_cast<const float4 *>(f.first + at));
            const float *q = f.rest + at;
            int k0 = 0;
            if (f.more <= kAtOnce / 4) {
                for (; k0 < f.more; ++k0) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(q + (int64_t)k0 * stride));
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
            }
            for (; k0 < f.more; k0 += kAtOnce) {
                float4 v[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    v[k] = k0 + k < f.more ? __ldcg(reinterpret_cast<const float4 *>(q + (int64_t)(k0 + k) * stride))
                                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
            }
            store_v(J, ((int64_t)f.tile * TM + row) * J.rank + c, c, row < f.rows ? f.used : 0, f.scale, s);
        }
    }
}

// ------------------------------------------------------------ expand
// y = base + W_i v of every tile, 128 columns a unit.  W_i [n x rank]
// (K-major: B_i) or [rank x n] (MN-major: A_i).  Persistent CTAs, each with a
// run of consecutive units (chunk fastest, so a tile's v stays).
struct ExpandJob {
    Rows base;
    CUtensorMap w, hi, lo, y;  // y: 32 rows x 64 columns
    int n, rank, mn, chunks;
    const int32_t *ranks;
    uint16_t *y_rows;
    int64_t ldy;
    int in_place;
};
struct ExpandParams {
    ExpandJob job[kMaxSiblings];
    int njobs, per_tile;  // chunks of a tile in all jobs
    int tokens;
    int behind_wgrad;  // wgrad is the launch before this one, and v older
    Plan plan;
    int *status;
};

constexpr int kExpandWarps = 8;  // of the epilogue
constexpr int kExpandThreads = 64 + 32 * (kExpandWarps + kLoaders - 1);
constexpr uint32_t kBaseBytes = TM * 256;  // 128 columns of a tile's rows: two halves of 64
constexpr uint32_t kVBytes = TM * 128;     // 64 columns of hi or lo
// NK: 64-wide blocks of the rank
template <int NK>
struct Expand {
    static constexpr int kStages = NK == 1 ? 4 : 2;
    static constexpr int kVBufs = 1;
    static constexpr uint32_t kW = NK * 2 * kBox;  // 128 columns x 64 NK
    static constexpr uint32_t kV = NK * 2 * kVBytes;
    static constexpr uint32_t kStage = kW + kBaseBytes;
    static constexpr size_t kSmem = 1024 + kVBufs * kV + kStages * kStage + 256;
};

template <int NK>
__global__ void __launch_bounds__(kExpandThreads, 1) expand_kernel(const __grid_constant__ ExpandParams p)
{
    using S = Expand<NK>;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t sV = base, sS = base + S::kVBufs * S::kV, bars = sS + S::kStages * S::kStage;
    const uint32_t full0 = bars, empty0 = full0 + 8 * S::kStages, accf0 = empty0 + 8 * S::kStages, acce0 = accf0 + 16;
    const uint32_t vfull0 = acce0 + 16, vempty0 = vfull0 + 16, drain = vempty0 + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (drain + 8 - raw));
    __shared__ int abort_shared;
    volatile int &abort_flag = abort_shared;

    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < S::kStages; ++s) {
                mbar_init(full0 + 8 * s, kFull);
                mbar_init(empty0 + 8 * s, kExpandWarps + 1);  // and the MMA thread
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(accf0 + 8 * b, 1);
                mbar_init(acce0 + 8 * b, kExpandWarps);
                mbar_init(vfull0 + 8 * b, 1);
                mbar_init(vempty0 + 8 * b, 1);
            }
            mbar_init(drain, 1);
            abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 256);
        tc_fence_before();
    } else if (warp == 0 && elect_one()) {
        for (int j = 0; j < p.njobs; ++j) {
            const ExpandJob &J = p.job[j];
            prefetch_map(&J.base.box);
            prefetch_map(&J.w);
            prefetch_map(&J.hi);
            prefetch_map(&J.lo);
            prefetch_map(&J.y);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Only v comes from the launch before; the plan was complete before that one
    // let this one start, and base and W are older still.  So the copies begin at
    // once, and loader 1, which fetches v, waits.  Behind wgrad v is older too:
    // this launch begins on the SMs that wgrad leaves, and only ends after it.
    const int ntiles = p.plan.counts[0];
    const int units = ntiles * p.per_tile;
    const int u0 = (int)((int64_t)units * blockIdx.x / gridDim.x), u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
    // Every role walks the same units, job by job, tile by tile.  What a unit
    // needs is in registers but where the tile changes (`fresh`): a parameter
    // read per unit and role costs as much as the unit's products.
    struct Walk {
        int job, tile, chunk, chunks;
        int kind;  // of the tile: 0 nothing to do, 1 copy base, 2 add
        Tile t;
        bool fresh;
    };
    auto enter = [&](Walk &q) {  // a new tile or job
        const ExpandJob &J = p.job[q.job];
        q.chunks = J.chunks;
        q.t = p.plan.tiles[q.tile];
        const int r = q.t.adapter >= 0 ? used_rank(J.ranks, J.rank, q.t.adapter) : 0;
        q.kind = r > 0 ? 2 : J.in_place ? 0 : 1;
        q.fresh = true;
    };
    auto start = [&]() {
        Walk q{};
        int r = u0;
        while (u0 < u1 && r >= p.job[q.job].chunks * ntiles) r -= p.job[q.job++].chunks * ntiles;
        if (u0 < u1) {
            q.tile = r / p.job[q.job].chunks;
            q.chunk = r - q.tile * p.job[q.job].chunks;
            enter(q);
        }
        return q;
    };
    auto advance = [&](Walk &q) {  // not past the last unit
        q.fresh = false;
        if (++q.chunk == q.chunks) {
            q.chunk = 0;
            if (++q.tile == ntiles) {
                q.tile = 0;
                ++q.job;
            }
            enter(q);
        }
    };

    const int loader = warp == 0 ? 0 : warp - 1 - kExpandWarps;
    if (warp == 0 || warp >= 2 + kExpandWarps) {
        int s = 0, nv = 0;
        uint32_t ph = 1;
        bool mn = false, run = false;
        const CUtensorMap *mb = nullptr, *mw = nullptr;
        int cols = 0;
        Copier<TM> mine;
        Walk q = start();
        for (int u = u0; u < u1; ++u) {  // to the end in every loader, whatever happens: they meet
            if (q.fresh && q.kind != 0) {
                const ExpandJob &J = p.job[q.job];
                mn = J.mn != 0;
                mb = &J.base.box;
                mw = &J.w;
                cols = J.base.cols;
                run = q.t.run();
                if (!run) {
                    mine.rows(J.base.p, J.base.ld, p.plan.perm + q.tile * TM, q.t.rows, 32 * loader + lane);
                    loaders_meet();  // the first is here, so nobody is ahead of the ring
                }
            }
            if (q.kind != 0) {
                const uint32_t dst = sS + s * S::kStage, bar = full0 + 8 * s;
                const int c0 = 128 * q.chunk;
                bool ok = true;
                if (loader == 0 || !run) {
                    ok = !abort_flag && mbar_wait(empty0 + 8 * s, ph);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) abort_flag = 1;
                }
                if (ok && loader == 0 && elect_one()) {
                    const uint32_t w_bytes = q.kind == 2 ? S::kW : 0u;
                    mbar_arrive_expect_tx(bar, w_bytes + (run ? kBaseBytes : 0u));
                    if (run) {
                        mbar_arrive_for_loaders(bar);
                        tma_load_2d(dst + S::kW, mb, c0, q.t.first, bar);
                        tma_load_2d(dst + S::kW + kBaseBytes / 2, mb, c0 + 64, q.t.first, bar);
                    }
                    if (q.kind == 2) {
#pragma unroll
                        for (int k = 0; k < NK; ++k) {
                            if (mn) {  // 64 rows of the rank x 128 columns
                                tma_load_3d(dst + (2 * k) * kBox, mw, c0, 64 * k, q.t.adapter, bar);
                                tma_load_3d(dst + (2 * k + 1) * kBox, mw, c0 + 64, 64 * k, q.t.adapter, bar);
                            } else {  // 128 rows x 64 columns of the rank
                                tma_load_3d(dst + k * 2 * kBox, mw, 64 * k, c0, q.t.adapter, bar);
                            }
                        }
                    }
                }
                __syncwarp();
                if (ok && !run) {
                    mine.copy<2>(dst + S::kW, kBaseBytes / 2, cols, c0, false);
                    mbar_arrive_after_copies(bar);
                }
                if (++s == S::kStages) s = 0, ph ^= 1;
            }
            if (loader == 1) {
                if (u == u0) {
                    if (!p.behind_wgrad) pdl_wait();
                    pdl_launch_dependents();
                }
                if (q.fresh && q.kind == 2) {
                    const ExpandJob &J = p.job[q.job];
                    const int b = nv % S::kVBufs;
                    const bool ok = !abort_flag && mbar_wait(vempty0 + 8 * b, ((uint32_t)(nv / S::kVBufs) & 1u) ^ 1u);
                    if (!__all_sync(0xffffffffu, ok)) {
                        abort_flag = 1;
                    } else if (elect_one()) {
                        const uint32_t bar = vfull0 + 8 * b, dst = sV + b * S::kV;
                        mbar_arrive_expect_tx(bar, S::kV);
                        for (int k = 0; k < NK; ++k) {
                            tma_load_2d(dst + (2 * k) * kVBytes, &J.hi, 64 * k, q.tile * TM, bar);
                            tma_load_2d(dst + (2 * k + 1) * kVBytes, &J.lo, 64 * k, q.tile * TM, bar);
                        }
                    }
                    __syncwarp();
                    ++nv;
                }
            }
            if (u + 1 < u1) advance(q);
        }
        if (loader == 1 && (u0 == u1 || p.behind_wgrad)) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if (abort_flag) drain_copies();
    } else if (warp == 1) {
        if (elect_one()) {
            int s = 0, nv = 0, na = 0, steps = 0;
            uint32_t ph = 0, idesc = 0, wstep = 0;
            uint32_t v0 = 0, wd0 = 0;
            Walk q = start();
            for (int u = u0; u < u1 && !abort_flag; ++u) {
                if (q.fresh && q.kind == 2) {
                    const ExpandJob &J = p.job[q.job];
                    const bool mn = J.mn != 0;
                    steps = (J.rank + 15) / 16;
                    idesc = idesc_of(128, false, mn);
                    wd0 = mn ? (uint32_t)smem_desc_mn(sS) : (uint32_t)smem_desc(sS);
                    wstep = mn ? 2048u >> 4 : 32u >> 4;
                    if (nv > 0) umma_commit(vempty0 + 8 * ((nv - 1) % S::kVBufs));  // the tile before is read
                    const int b = nv % S::kVBufs;
                    if (!mbar_wait(vfull0 + 8 * b, (uint32_t)(nv / S::kVBufs) & 1u)) {
                        abort_flag = 1;
                        break;
                    }
                    v0 = (uint32_t)smem_desc(sV + b * S::kV);
                    ++nv;
                }
                // A stage's phases are all waited for, with a product or without, and the
                // stage is given back by this thread too: where base is only copied nothing
                // else keeps the ring from turning past it.
                if (q.kind != 0) {
                    const int ab = na & 1;
                    if ((q.kind == 2 && !mbar_wait(acce0 + 8 * ab, ((uint32_t)(na >> 1) & 1u) ^ 1u)) ||
                        !mbar_wait(full0 + 8 * s, ph) || abort_flag) {
                        abort_flag = 1;
                        break;
                    }
                    if (q.kind == 2) {
                        tc_fence_after();
                        const uint32_t acc = tmem + 128 * ab, at = (uint32_t)s * (S::kStage >> 4);
#pragma unroll
                        for (int i = 0; i < 4 * NK; ++i) {
                            if (i < steps) {
                                const uint32_t w = wd0 + at + (i >> 2) * (2 * kBox >> 4) + (i & 3) * wstep;
                                const uint32_t v = v0 + (i >> 2) * (2 * kVBytes >> 4) + (i & 3) * 2;
                                umma_lo(acc, v, w, idesc, i != 0 ? 1u : 0u);
                                umma_lo(acc, v + (kVBytes >> 4), w, idesc, 1u);
                            }
                        }
                        umma_commit(accf0 + 8 * ab);
                        ++na;
                    }
                    mbar_arrive(empty0 + 8 * s);  // the epilogue's arrivals come after the products
                    if (++s == S::kStages) s = 0, ph ^= 1;
                }
                if (u + 1 < u1) advance(q);
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else {
        // epilogue: warp e takes rows 32 (warp % 4) .. and 64 of the unit's columns
        const int quad = warp & 3, half = (warp - 2) >> 2, row = 32 * quad + lane, tokens = p.tokens;
        // 32 consecutive rows go back as one box, others a row of 128 bytes
        // for each 8 lanes.  A box is read from the stage in the background, so
        // the stage is given back a unit later.
        int s = 0, na = 0, tok = 0, n = 0, held = -1;
        uint32_t ph = 0;
        uint16_t *to[8];  // where this lane's columns of the job go
        bool run = false;
        int row0 = 0;
        const CUtensorMap *my = nullptr;
        Walk q = start();
        for (int u = u0; u < u1; ++u) {
            if (q.fresh) {
                const ExpandJob &J = p.job[q.job];
                tok = p.plan.perm[q.tile * TM + row];
                row0 = __shfl_sync(0xffffffffu, tok, 0);
                run = __all_sync(0xffffffffu, tok < tokens && tok == row0 + lane);
                my = &J.y;
                n = J.n;
                if (!run) {
                    uint16_t *y = J.y_rows + 64 * half + 8 * (lane & 7);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = __shfl_sync(0xffffffffu, tok, 4 * i + (lane >> 3));
                        to[i] = t < tokens ? y + t * J.ldy : nullptr;
                    }
                }
            }
            if (q.kind == 0) {
                if (u + 1 < u1) advance(q);
                continue;
            }
            const int ab = na & 1;
            bool ok = !abort_flag && mbar_wait(full0 + 8 * s, ph);
            if (ok && q.kind == 2) ok = mbar_wait(accf0 + 8 * ab, (uint32_t)(na >> 1) & 1u);
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            const uint32_t tile = sS + s * S::kStage + S::kW + (uint32_t)half * (kBaseBytes / 2);
            if (q.kind == 2) {
                tc_fence_after();
                const uint32_t at = tile + (uint32_t)row * 128u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 b[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) b[c] = ld_shared_v4(at + (uint32_t)(((4 * h + c) ^ (row & 7)) << 4));
                    uint32_t v[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * ab + 64 * half + 32 * h), v);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        b[c].x = add_bf162(b[c].x, v[8 * c], v[8 * c + 1]);
                        b[c].y = add_bf162(b[c].y, v[8 * c + 2], v[8 * c + 3]);
                        b[c].z = add_bf162(b[c].z, v[8 * c + 4], v[8 * c + 5]);
                        b[c].w = add_bf162(b[c].w, v[8 * c + 6], v[8 * c + 7]);
                        st_shared_v4(at + (uint32_t)(((4 * h + c) ^ (row & 7)) << 4), b[c]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * ab);
                ++na;
            }
            const int c0 = 128 * q.chunk;
            fence_async_shared();  // for the box, and for the next copy into this stage
            __syncwarp();
            if (run) {
                if (lane == 0) {
                    if (c0 + 64 * half < n) tma_store_2d(my, c0 + 64 * half, row0, tile + (uint32_t)quad * 4096u);
                    bulk_commit();
                    if (S::kStages > 2) {
                        bulk_wait_read<1>();
                        if (held >= 0) mbar_arrive(empty0 + 8 * held);
                        held = s;
                    } else {  // none to spare
                        bulk_wait_read<0>();
                        mbar_arrive(empty0 + 8 * s);
                    }
                }
            } else {
                const bool in = c0 + 64 * half + 8 * (lane & 7) < n;
                uint4 o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int tr = 32 * quad + 4 * i + (lane >> 3);
                    o[i] = ld_shared_v4(tile + (uint32_t)tr * 128u + (uint32_t)(((lane & 7) ^ (tr & 7)) << 4));
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if (held >= 0) {
                        bulk_wait_read<0>();
                        mbar_arrive(empty0 + 8 * held);
                        held = -1;
                    }
                    mbar_arrive(empty0 + 8 * s);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (to[i] != nullptr && in) *reinterpret_cast<uint4 *>(to[i] + c0) = o[i];
            }
            if (++s == S::kStages) s = 0, ph ^= 1;
            if (u + 1 < u1) advance(q);
        }
        if (lane == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) set_status(p.status, LB_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ------------------------------------------------------------ wgrad
// dA_i[r][n] = sum over an adapter's slots of u[slot][r] x[slot][n], and dB_i
// the same of v and dy with the result [n][r]: D[n][r] with the slots as K, both
// operands MN-major (slots outermost), 64 slots a K-block.  A product is kCols
// columns n of one adapter: with ranks up to 64 two MMA tiles, so that v, three
// bf16 parts wide, comes from L2 half as often for the x it meets (a tile alone
// moved 40 KB for 16 KB of x and took 108 us at 8192 tokens).  Shares as in
// shrink, adapter by adapter.
struct WgradJob {
    Rows x;
    CUtensorMap v[kParts];
    int n, products;  // columns; products of an adapter
    int transposed;   // the gradient is [r][n]
    float *out;       // [adapter][...]
};
struct AdapterWgradParams {
    WgradJob job[2];
    int rank, count, ctas;
    const int32_t *ranks;
    Plan plan;
    float *part;  // [slot][kCols * rank], the gradient's order
    int *status;
};

constexpr int kWgradWarps = 8;  // of the epilogue
constexpr int kWgradThreads = 64 + 32 * (kWgradWarps + kLoaders - 1);
template <int NK>
struct Wgrad {
    static constexpr int kTiles = NK == 1 ? 2 : 1;  // of 128 columns
    static constexpr int kCols = 128 * kTiles;
    static constexpr uint32_t kX = kTiles * 2 * kBox;
    static constexpr uint32_t kStage = kX + kParts * NK * kBox;
    static constexpr int kStages = NK == 1 ? 4 : 3;
    static constexpr size_t kSmem = 1024 + kStages * kStage + 256;
};

// The product at K-block w of all the work: adapter i has block0[i] .. blocks,
// each of them `per` (products of both jobs) times.  From one product to the
// next nothing is read but where the adapter changes: a search for each left
// the copies idle for two microseconds.
template <int NK>
struct Product {
    const AdapterWgradParams &p;
    int per, job0, adapter, m, job, n0, begin, nkb, kb, tile0;
    Tile first;  // the adapter's first tile
    __device__ __forceinline__ Product(const AdapterWgradParams &params, int w, bool any) : p(params)
    {
        if (!any) return;  // a CTA without a share
        job0 = p.job[0].products;
        per = job0 + p.job[1].products;
        int lo = 0, hi = p.count;  // the last adapter with block0 * per <= w (those without blocks come before it)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.plan.block0[mid] * per <= w)
                lo = mid;
            else
                hi = mid;
        }
        adapter = lo;
        const int b0 = enter();
        m = (w - b0) / nkb;
        begin = b0 + m * nkb;
        kb = w - begin;
        locate();
    }
    __device__ __forceinline__ int enter()
    {
        const int b0 = p.plan.block0[adapter];
        nkb = p.plan.block0[adapter + 1] - b0;
        tile0 = p.plan.tile0[adapter];
        first = p.plan.tiles[tile0];
        return b0 * per;
    }
    __device__ __forceinline__ void locate()
    {
        job = m >= job0;
        n0 = Wgrad<NK>::kCols * (job ? m - job0 : m);
    }
    __device__ __forceinline__ void advance()  // not past the last one
    {
        begin += nkb;
        kb = 0;
        if (++m == per) {
            m = 0;
            do {
                ++adapter;
                enter();
            } while (nkb == 0);
        }
        locate();
    }
};

template <int NK>
__global__ void __launch_bounds__(kWgradThreads, 1) adapter_wgrad_kernel(const __grid_constant__ AdapterWgradParams p)
{
    using S = Wgrad<NK>;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t bars = base + S::kStages * S::kStage;
    const uint32_t full0 = bars, empty0 = full0 + 8 * S::kStages, accf0 = empty0 + 8 * S::kStages, acce0 = accf0 + 16;
    const uint32_t drain = acce0 + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (drain + 8 - raw));
    __shared__ int abort_shared;
    volatile int &abort_flag = abort_shared;

    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < S::kStages; ++s) {
                mbar_init(full0 + 8 * s, kFull);
                mbar_init(empty0 + 8 * s, 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(accf0 + 8 * b, 1);
                mbar_init(acce0 + 8 * b, kWgradWarps);
            }
            mbar_init(drain, 1);
            abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), 512);
        tc_fence_before();
    } else if (warp == 0 && elect_one()) {
        for (int j = 0; j < 2; ++j) {
            prefetch_map(&p.job[j].x.box);
            for (int i = 0; i < kParts; ++i) prefetch_map(p.job[j].v + i);
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Only v comes from the launch before: as in expand, the other copies begin
    // at once, and loader 1, which fetches v, waits.

    const int cta = blockIdx.x;
    const Shares shares(p.plan.counts[2] * (p.job[0].products + p.job[1].products), p.ctas, 1);
    const int w0 = cta < shares.ctas ? shares.start(cta) : 0, w1 = cta < shares.ctas ? shares.start(cta + 1) : 0;

    const int loader = warp == 0 ? 0 : warp - 1 - kWgradWarps;
    if (warp == 0 || warp >= 2 + kWgradWarps) {
        int s = 0;
        uint32_t ph = 1;
        Product<NK> q(p, w0, w0 < w1);
        bool waited = false;
        // Loaders 2 and 3 take no part in a box, so the ring turns without them
        // there and the parity they would wait for may come round again: they leave
        // such K-blocks alone, and all loaders meet at the next one of copies, so
        // that nobody is a turn ahead of the ring or behind it.
        bool boxes = false;  // since they last met
        for (int w = w0; w < w1;) {  // to the end in every loader, whatever happens: they meet
            const int n = min(q.nkb - q.kb, w1 - w);
            const WgradJob &J = p.job[q.job];
            const CUtensorMap *mx = &J.x.box, *mv = J.v;
            const uint16_t *x = J.x.p;
            const int64_t ld = J.x.ld;
            const int tile0 = q.tile0, end = q.kb + n;
            Tile T = q.first;
            if (q.kb >= 2) T = p.plan.tiles[tile0 + q.kb / 2];
            Tile next = T;
            Copier<64> mine, ahead;
            auto find = [&](Copier<64> &c, const Tile &t, int kb) {  // the rows of a K-block that is no box
                const int left = t.rows - 64 * (kb & 1);
                if (t.run() && left < 64) c.run(x, ld, t.first + 64 * (kb & 1), left, 32 * loader + lane);
                if (!t.run()) c.rows(x, ld, p.plan.perm + tile0 * TM + 64 * kb, left, 32 * loader + lane);
            };
            find(mine, T, q.kb);
            for (int kb = q.kb; kb < end; ++kb) {
                const int half = kb & 1;
                if (half == 0) T = next;
                if (half == 0 || kb == q.kb) {  // ahead of use
                    if ((kb | 1) + 1 < end) next = p.plan.tiles[tile0 + kb / 2 + 1];
                }
                if (kb + 1 < end) find(ahead, half == 0 ? T : next, kb + 1);
                const uint32_t dst = base + s * S::kStage, bar = full0 + 8 * s;
                const int slot = tile0 * TM + 64 * kb;
                const bool run = T.run() && T.rows >= 64 * half + 64;
                if (!run && boxes) loaders_meet();
                boxes = run;
                bool ok = true;
                if (!run || loader < 2) {
                    ok = !abort_flag && mbar_wait(empty0 + 8 * s, ph);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) abort_flag = 1;
                }
                if (ok && loader == 0 && elect_one()) {
                    mbar_arrive_expect_tx(bar, S::kStage - (run ? 0u : S::kX));
                    if (run) {
                        mbar_arrive_for_loaders(bar);
#pragma unroll
                        for (int c = 0; c < 2 * S::kTiles; ++c)
                            tma_load_2d(dst + c * kBox, mx, q.n0 + 64 * c, T.first + 64 * half, bar);
                    }
                }
                __syncwarp();
                if (ok && !run) {  // zeros past the adapter's tokens: the slots are what is summed over
                    mine.copy<2 * S::kTiles>(dst, kBox, J.x.cols, q.n0, true);
                    mbar_arrive_after_copies(bar);
                }
                if (loader == 1) {
                    if (!waited) {
                        waited = true;
                        pdl_wait();
                        pdl_launch_dependents();
                    }
                    if (ok && elect_one()) {
#pragma unroll
                        for (int i = 0; i < kParts; ++i)
#pragma unroll
                            for (int k = 0; k < NK; ++k)
                                tma_load_2d(dst + S::kX + (i * NK + k) * kBox, mv + i, 64 * k, slot, bar);
                    }
                    __syncwarp();
                }
                mine = ahead;
                if (++s == S::kStages) s = 0, ph ^= 1;
            }
            w += n;
            if (w < w1) q.advance();
        }
        if (loader == 1 && !waited) {
            pdl_wait();
            pdl_launch_dependents();
        }
        if (abort_flag) drain_copies();
    } else if (warp == 1) {
        if (elect_one()) {
            // v's parts side by side as N, so that x is read less often from
            // shared memory: the first two, then the third onto the second's sums
            constexpr int NH = 64 * NK;
            const uint32_t idesc = idesc_of(2 * NH, true, true), idesc2 = idesc_of(NH, true, true);
            const uint32_t a0 = (uint32_t)smem_desc_mn(base), b0 = (uint32_t)smem_desc_mn(base + S::kX);
            int s = 0, na = 0;  // stage; segments so far
            uint32_t ph = 0;
            Product<NK> q(p, w0, w0 < w1);
            for (int w = w0; w < w1 && !abort_flag;) {
                const int n = min(q.nkb - q.kb, w1 - w);
                for (int i = 0; i < n; ++i) {
                    const int ab = na & 1;
                    const bool first = i % kSegment == 0;
                    if ((first && !mbar_wait(acce0 + 8 * ab, ((uint32_t)(na >> 1) & 1u) ^ 1u)) ||
                        !mbar_wait(full0 + 8 * s, ph) || abort_flag) {
                        abort_flag = 1;
                        break;
                    }
                    fence_async_shared();  // the loaders' writes, before the MMA reads them
                    tc_fence_after();
                    const uint32_t at = (uint32_t)s * (S::kStage >> 4), acc = tmem + 256 * ab;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t bd = b0 + at + kk * (2048u >> 4);
#pragma unroll
                        for (int m = 0; m < S::kTiles; ++m) {
                            const uint32_t ad = a0 + at + m * (2 * kBox >> 4) + kk * (2048u >> 4);
                            umma_lo(acc + 128 * m, ad, bd, idesc, !first || kk != 0 ? 1u : 0u);
                            umma_lo(acc + 128 * m + NH, ad, bd + (2 * NK * kBox >> 4), idesc2, 1u);
                        }
                    }
                    umma_commit(empty0 + 8 * s);
                    if (i % kSegment == kSegment - 1 || i + 1 == n) {
                        umma_commit(accf0 + 8 * ab);
                        ++na;
                    }
                    if (++s == S::kStages) s = 0, ph ^= 1;
                }
                w += n;
                if (w < w1) q.advance();
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else {
        // a column n a lane, 64 of the rank: warps 2 .. 5 and 6 .. 9 take the
        // two tiles (NK = 1), or the two halves of the rank
        const int quad = warp & 3, part = (warp - 2) >> 2;
        const int n_local = 32 * quad + lane + (NK == 1 ? 128 * part : 0), c0 = NK == 1 ? 0 : 64 * part;
        const uint32_t lane_at = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(NK == 1 ? 128 * part : 64 * part);
        const int nr = min(64, ((p.rank + 15) & ~15) - c0);
        int na = 0;
        Product<NK> q(p, w0, w0 < w1);
        for (int w = w0; w < w1;) {
            const int n = min(q.nkb - q.kb, w1 - w);
            float sum[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) sum[c] = 0.0f;
            bool ok = true;
            for (int i = 0; i < n; i += kSegment, ++na) {
                const int ab = na & 1;
                ok = !abort_flag && mbar_wait(accf0 + 8 * ab, (uint32_t)(na >> 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    if (c < nr) {
                        uint32_t v[16], r[16];
                        tmem_ld16(lane_at + (uint32_t)(256 * ab + c), v);
                        tmem_ld16(lane_at + (uint32_t)(256 * ab + 64 * NK + c), r);
#pragma unroll
                        for (int e = 0; e < 16; ++e) sum[c + e] += __uint_as_float(v[e]) + __uint_as_float(r[e]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * ab);
            }
            if (!ok) {
                abort_flag = 1;
                break;
            }
            w += n;
            const WgradJob &J = p.job[q.job];
            const bool whole = n == q.nkb;
            const int used = whole ? used_rank(p.ranks, p.rank, q.adapter) : p.rank;
            // its place in the gradient, or among the shared sums
            float *out = whole ? J.out + (int64_t)q.adapter * p.rank * J.n
                               : p.part + (int64_t)shares.slot(cta, q.begin) * S::kCols * p.rank;
            const int col = (whole ? q.n0 : 0) + n_local, ld = whole ? J.n : S::kCols;
            if (q.n0 + n_local < J.n) {  // uniform over the warp
                if (J.transposed) {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (c0 + c < p.rank) out[(int64_t)(c0 + c) * ld + col] = c0 + c < used ? sum[c] : 0.0f;
                } else {
#pragma unroll
                    for (int c = 0; c < 64; c += 4)
                        if (c0 + c < p.rank)
                            *reinterpret_cast<float4 *>(out + (int64_t)col * p.rank + c0 + c) =
                                make_float4(c0 + c < used ? sum[c] : 0.0f, c0 + c + 1 < used ? sum[c + 1] : 0.0f,
                                            c0 + c + 2 < used ? sum[c + 2] : 0.0f, c0 + c + 3 < used ? sum[c + 3] : 0.0f);
                }
            }
            if (w < w1) q.advance();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (abort_flag && threadIdx.x == 0) set_status(p.status, LB_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The products of wgrad that several CTAs share, and zeros for adapters that no
// token uses; 1024 quads of the gradient a unit.
constexpr int kQuads = 1024;
template <int NK>
__global__ void __launch_bounds__(kFinishThreads) wgrad_finish_kernel(const __grid_constant__ AdapterWgradParams p)
{
    constexpr int kCols = Wgrad<NK>::kCols;
    struct Found {
        int adapter, job, n0, i0, used, sums;  // sums: shared sums, -1 nothing to do
        const float *first, *rest;
    };
    __shared__ Found found;
    const int per = p.job[0].products + p.job[1].products;
    const int quads = kCols * p.rank / 4, each = (quads + kQuads - 1) / kQuads, units = p.count * per * each;
    auto find = [&](int u) {  // by the plan, as in shrink's finish
        if (threadIdx.x == 0 && u < units) {
            const int product = u / each, adapter = product / per, m = product - adapter * per;
            const int b0 = p.plan.block0[adapter], nkb = p.plan.block0[adapter + 1] - b0;
            found.sums = 0;
            if (nkb > 0) {
                const Shares shares(p.plan.counts[2] * per, p.ctas, 1);
                const int begin = b0 * per + m * nkb;
                const int first = shares.owner(begin), last = shares.owner(begin + nkb - 1);
                found.sums = last > first ? last - first + 1 : -1;
                found.first = p.part + (int64_t)shares.slot(first, begin) * 4 * quads;
                found.rest = p.part + (int64_t)2 * (first + 1) * 4 * quads;
            }
            found.adapter = adapter;
            found.job = m >= p.job[0].products;
            found.n0 = kCols * (found.job ? m - p.job[0].products : m);
            found.i0 = (u - product * each) * kQuads;
            found.used = used_rank(p.ranks, p.rank, adapter);
        }
    };
    find(blockIdx.x);
    pdl_wait();
    pdl_launch_dependents();
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        __syncthreads();
        const Found f = found;
        __syncthreads();
        find(u + gridDim.x);
        if (f.sums < 0) continue;
        const WgradJob &J = p.job[f.job];
        const int N = J.n, used = f.used, cols = p.rank / 4, transposed = J.transposed;
        float *out = J.out + (int64_t)f.adapter * p.rank * N + (transposed ? f.n0 : (int64_t)f.n0 * p.rank);
#pragma unroll
        for (int j = 0; j < kQuads / kFinishThreads; ++j) {
            const int i = f.i0 + j * kFinishThreads + threadIdx.x;
            if (i >= quads) break;
            const int q = transposed ? i / (kCols / 4) : i / cols;  // r, or n
            const int n = transposed ? 4 * (i - q * (kCols / 4)) : q, c = transposed ? q : 4 * (i - q * cols);
            if (f.n0 + n >= N) continue;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (f.sums > 0) {
                s = __ldcg(reinterpret_cast<const float4 *>(f.first) + i);
#pragma unroll 4
                for (int k = 0; k < f.sums - 1; ++k) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(f.rest) + (int64_t)k * 2 * quads + i);
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
            }
            // zeros past the adapter's rank
            const int left = transposed ? (c < used ? 4 : 0) : used - c;
            s = make_float4(left > 0 ? s.x : 0.0f, left > 1 ? s.y : 0.0f, left > 2 ? s.z : 0.0f, left > 3 ? s.w : 0.0f);
            *reinterpret_cast<float4 *>(out + (transposed ? (int64_t)c * N + n : (int64_t)n * p.rank + c)) = s;
        }
    }
}

// ------------------------------------------------------------ host side
size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

constexpr int kMostCtas = 148;  // of shrink and wgrad, whatever the device has: workspaces are sized by it

// Tiles of a batch: at most one partial tile per adapter in use, and for the
// tokens without one.
int most_tiles(int tokens, int count) { return tokens / TM + std::min(count + 1, tokens); }

struct Layout {
    size_t counts, tiles, perm, block0, tile0, v[kMaxSiblings][kParts], sums, grads, total;
};
// nv: products v per tile, of `parts` bf16 each; grad_floats: of the shared sums of wgrad
Layout layout_of(int tokens, int count, int nv, const int *ranks, int parts, size_t grad_floats)
{
    Layout L{};
    size_t off = 0;
    const size_t tiles = (size_t)most_tiles(tokens, count);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += align256(bytes);
        return at;
    };
    L.counts = take(4 * sizeof(int));
    L.tiles = take(tiles * sizeof(Tile));
    L.perm = take(tiles * TM * sizeof(int));
    L.block0 = take((size_t)(count + 1) * sizeof(int));
    L.tile0 = take((size_t)count * sizeof(int));
    int widest = 0;
    for (int j = 0; j < nv; ++j) widest = std::max(widest, ranks[j]);
    L.sums = take((size_t)2 * kMostCtas * TM * (size_t)widest * sizeof(float));
    for (int j = 0; j < nv; ++j)
        for (int q = 0; q < parts; ++q) L.v[j][q] = take(tiles * TM * (size_t)ranks[j] * 2);
    L.grads = take(grad_floats * sizeof(float));
    L.total = off;
    return L;
}

Plan plan_at(const Layout &L, uint8_t *ws)
{
    Plan p;
    p.counts = reinterpret_cast<int *>(ws + L.counts);
    p.tiles = reinterpret_cast<Tile *>(ws + L.tiles);
    p.perm = reinterpret_cast<int *>(ws + L.perm);
    p.block0 = reinterpret_cast<int *>(ws + L.block0);
    p.tile0 = reinterpret_cast<int *>(ws + L.tile0);
    return p;
}

cudaError_t encode_rows(Rows *m, const uint16_t *ptr, int rows, int cols, int64_t ld, int box)
{
    m->p = ptr;
    m->ld = ld;
    m->cols = cols;
    return encode_2d(&m->box, ptr, rows, cols, ld, true, box);
}
// A dense bf16 [n2][n1][n0] in boxes of box1 x 64.
cudaError_t encode_3d(CUtensorMap *tm, const void *ptr, int n0, int n1, int n2, int box1)
{
    PFN_cuTensorMapEncodeTiled_v12000 encode = encoder_slot();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)n0 * 2, (cuuint64_t)n0 * (cuuint64_t)n1 * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box1, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename K, typename P>
cudaError_t launch(K kernel, int grid, int threads, size_t smem, const P &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_plan(const int32_t *ids, int tokens, int count, const Plan &plan, const DeviceInfo &dev, cudaStream_t stream)
{
    const PlanParams p{ids, tokens, count, plan, dev.status};
    return launch(plan_kernel, 1, kPlanThreads, sizeof(int) * kPlanWarps * (size_t)(count + 1), p, stream);
}

cudaError_t launch_shrink(ShrinkParams &p, int tiles, const DeviceInfo &dev, cudaStream_t stream)
{
    p.ctas = std::min(dev.sm_count, kMostCtas);
    const cudaError_t e = p.part_rank <= 64 ? launch(shrink_kernel<1>, p.ctas, kShrinkThreads, Shrink<1>::kSmem, p, stream)
                                            : launch(shrink_kernel<2>, p.ctas, kShrinkThreads, Shrink<2>::kSmem, p, stream);
    return e != cudaSuccess ? e : launch(shrink_finish_kernel, std::min(tiles * p.njobs * (TM / kFinishRows), 16 * dev.sm_count), kFinishThreads,
                                        0, p, stream);
}

template <int NK>
cudaError_t launch_wgrad(AdapterWgradParams &p, const DeviceInfo &dev, cudaStream_t stream)
{
    for (WgradJob &J : p.job) J.products = (J.n + Wgrad<NK>::kCols - 1) / Wgrad<NK>::kCols;
    p.ctas = std::min(dev.sm_count, kMostCtas);
    return launch(adapter_wgrad_kernel<NK>, p.ctas, kWgradThreads, Wgrad<NK>::kSmem, p, stream);
}
size_t wgrad_shared_floats(int rank)
{
    return (size_t)2 * kMostCtas * (size_t)(rank <= 64 ? Wgrad<1>::kCols : Wgrad<2>::kCols) * (size_t)rank;
}

cudaError_t launch_expand(const ExpandParams &p, int rank, const DeviceInfo &dev, cudaStream_t stream)
{
    return rank <= 64 ? launch(expand_kernel<1>, dev.sm_count, kExpandThreads, Expand<1>::kSmem, p, stream)
                      : launch(expand_kernel<2>, dev.sm_count, kExpandThreads, Expand<2>::kSmem, p, stream);
}

}  // namespace

cudaError_t adapters_mma_prepare_device(const DeviceInfo &dev)
{
    (void)dev;
    cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(int) * kPlanWarps * (LB_MAX_ADAPTERS + 1)));
    auto allow = [&](auto kernel, size_t bytes) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    };
    allow(shrink_kernel<1>, Shrink<1>::kSmem);
    allow(shrink_kernel<2>, Shrink<2>::kSmem);
    allow(expand_kernel<1>, Expand<1>::kSmem);
    allow(expand_kernel<2>, Expand<2>::kSmem);
    allow(adapter_wgrad_kernel<1>, Wgrad<1>::kSmem);
    allow(adapter_wgrad_kernel<2>, Wgrad<2>::kSmem);
    return e;
}

size_t adapters_mma_workspace_bytes(int tokens, int count, int nproj, const int *ranks)
{
    return layout_of(tokens, count, nproj, ranks, 2, 0).total;
}

cudaError_t adapters_mma_forward(const AdaptersArgs &a, const DeviceInfo &dev, cudaStream_t stream)
{
    cudaError_t e = get_encoder();
    if (e != cudaSuccess) return e;
    int ranks[kMaxSiblings], widest = 0;
    for (int j = 0; j < a.nproj; ++j) {
        ranks[j] = a.proj[j].rank;
        widest = std::max(widest, ranks[j]);
    }
    const Layout L = layout_of(a.tokens, a.count, a.nproj, ranks, 2, 0);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const Plan plan = plan_at(L, ws);
    const int tiles = most_tiles(a.tokens, a.count);
    ShrinkParams sp{};
    ExpandParams ep{};
    sp.plan = ep.plan = plan;
    sp.status = ep.status = dev.status;
    ep.njobs = a.nproj;
    ep.tokens = a.tokens;
    Rows mx;
    e = encode_rows(&mx, a.x, a.tokens, a.n_in, a.ldx, TM);
    for (int j = 0; j < a.nproj && e == cudaSuccess; ++j) {
        const AdapterProj &P = a.proj[j];
        ShrinkJob &s = sp.job[j];
        s.x = mx;
        s.nkb = (a.n_in + 63) / 64;
        sp.per_tile += s.nkb;
        s.rank = P.rank;
        s.ranks = P.ranks;
        s.scale = P.scale;
        for (int q = 0; q < 2; ++q) s.v[q] = reinterpret_cast<uint16_t *>(ws + L.v[j][q]);
        e = encode_3d(&s.w, P.a, a.n_in, P.rank, a.count, (P.rank + 15) & ~15);
        ExpandJob &x = ep.job[j];
        x.n = P.n_out;
        x.rank = P.rank;
        x.chunks = (P.n_out + 127) / 128;
        ep.per_tile += x.chunks;
        x.ranks = P.ranks;
        x.y_rows = P.y;
        x.ldy = P.ldy;
        x.in_place = P.base == P.y;
        if (e == cudaSuccess) e = encode_rows(&x.base, P.base, a.tokens, P.n_out, P.ldbase, TM);
        if (e == cudaSuccess) e = encode_2d(&x.y, P.y, a.tokens, P.n_out, P.ldy, true, 32);
        if (e == cudaSuccess) e = encode_3d(&x.w, P.b, P.rank, P.n_out, a.count, 128);
        if (e == cudaSuccess) e = encode_2d(&x.hi, s.v[0], tiles * TM, P.rank, P.rank, true, TM);
        if (e == cudaSuccess) e = encode_2d(&x.lo, s.v[1], tiles * TM, P.rank, P.rank, true, TM);
    }
    sp.njobs = a.nproj;
    sp.part = reinterpret_cast<float *>(ws + L.sums);
    sp.part_rank = widest;
    if (e == cudaSuccess) e = launch_plan(a.ids, a.tokens, a.count, plan, dev, stream);
    if (e == cudaSuccess) e = launch_shrink(sp, tiles, dev, stream);
    if (e == cudaSuccess) e = launch_expand(ep, widest, dev, stream);
    return e;
}

size_t adapters_mma_backward_workspace_bytes(int tokens, int count, int rank)
{
    const int ranks[2] = {rank, rank};
    return layout_of(tokens, count, 2, ranks, kParts, wgrad_shared_floats(rank)).total;
}

cudaError_t adapters_mma_backward(const AdaptersBwdArgs &b, const DeviceInfo &dev, cudaStream_t stream)
{
    cudaError_t e = get_encoder();
    if (e != cudaSuccess) return e;
    const int ranks[2] = {b.rank, b.rank};
    const Layout L = layout_of(b.tokens, b.count, 2, ranks, kParts, wgrad_shared_floats(b.rank));
    uint8_t *ws = static_cast<uint8_t *>(b.workspace);
    const Plan plan = plan_at(L, ws);
    const int tiles = most_tiles(b.tokens, b.count);
    uint16_t *v[2][kParts];  // v, then u
    Rows mx, mdy;
    CUtensorMap mhi, mlo;
    for (int q = 0; q < 2; ++q)
        for (int i = 0; i < kParts; ++i) v[q][i] = reinterpret_cast<uint16_t *>(ws + L.v[q][i]);
    e = encode_2d(&mhi, v[1][0], tiles * TM, b.rank, b.rank, true, TM);
    if (e == cudaSuccess) e = encode_2d(&mlo, v[1][1], tiles * TM, b.rank, b.rank, true, TM);
    if (e == cudaSuccess) e = encode_rows(&mx, b.x, b.tokens, b.n_in, b.ldx, TM);
    if (e == cudaSuccess) e = encode_rows(&mdy, b.dy, b.tokens, b.n_out, b.lddy, TM);
    ShrinkParams sp{};
    sp.plan = plan;
    sp.status = dev.status;
    for (int q = 0; q < 2; ++q) {
        ShrinkJob &s = sp.job[q];
        s.x = q ? mdy : mx;
        s.nkb = ((q ? b.n_out : b.n_in) + 63) / 64;
        sp.per_tile += s.nkb;
        s.rank = b.rank;
        s.mn = q;
        s.ranks = b.ranks;
        s.scale = b.scale;
        for (int i = 0; i < kParts; ++i) s.v[i] = v[q][i];
    }
    if (e == cudaSuccess) e = encode_3d(&sp.job[0].w, b.a, b.n_in, b.rank, b.count, (b.rank + 15) & ~15);
    if (e == cudaSuccess) e = encode_3d(&sp.job[1].w, b.b, b.rank, b.n_out, b.count, 64);
    sp.njobs = 2;
    sp.part = reinterpret_cast<float *>(ws + L.sums);
    sp.part_rank = b.rank;
    if (e == cudaSuccess) e = launch_plan(b.ids, b.tokens, b.count, plan, dev, stream);
    if (e == cudaSuccess) e = launch_shrink(sp, tiles, dev, stream);
    AdapterWgradParams wp{};
    wp.rank = b.rank;
    wp.count = b.count;
    wp.ranks = b.ranks;
    wp.plan = plan;
    wp.part = reinterpret_cast<float *>(ws + L.grads);
    wp.status = dev.status;
    for (int q = 0; q < 2; ++q) {  // dA from x and u, dB from dy and v
        WgradJob &w = wp.job[q];
        w.x = q ? mdy : mx;
        if (e == cudaSuccess)
            e = encode_2d(&w.x.box, q ? b.dy : b.x, b.tokens, q ? b.n_out : b.n_in, q ? b.lddy : b.ldx, true, 64);
        for (int i = 0; i < kParts && e == cudaSuccess; ++i)
            e = encode_2d(&w.v[i], v[1 - q][i], tiles * TM, b.rank, b.rank, true, 64);
        w.n = q ? b.n_out : b.n_in;
        w.transposed = !q;
        w.out = q ? b.db : b.da;
    }
    if (e == cudaSuccess) e = b.rank <= 64 ? launch_wgrad<1>(wp, dev, stream) : launch_wgrad<2>(wp, dev, stream);
    if (b.dx != nullptr && e == cudaSuccess) {
        ExpandParams ep{};
        ep.plan = plan;
        ep.behind_wgrad = 1;
        ep.status = dev.status;
        ep.njobs = 1;
        ep.tokens = b.tokens;
        ExpandJob &x = ep.job[0];
        x.n = b.n_in;
        x.rank = b.rank;
        x.mn = 1;
        x.chunks = ep.per_tile = (b.n_in + 127) / 128;
        x.ranks = b.ranks;
        x.y_rows = b.dx;
        x.ldy = b.lddx;
        x.in_place = b.dx_base == b.dx;
        x.hi = mhi;
        x.lo = mlo;
        e = encode_rows(&x.base, b.dx_base, b.tokens, b.n_in, b.lddxbase, TM);
        if (e == cudaSuccess) e = encode_2d(&x.y, b.dx, b.tokens, b.n_in, b.lddx, true, 32);
        if (e == cudaSuccess) e = encode_3d(&x.w, b.a, b.n_in, b.rank, b.count, 64);
        if (e == cudaSuccess) e = launch_expand(ep, b.rank, dev, stream);
    }
    if (e != cudaSuccess) return e;
    return b.rank <= 64 ? launch(wgrad_finish_kernel<1>, 8 * dev.sm_count, kFinishThreads, 0, wp, stream)
                        : launch(wgrad_finish_kernel<2>, 8 * dev.sm_count, kFinishThreads, 0, wp, stream);
}

}  // namespace lb
