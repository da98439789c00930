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
//   shrink  a tile's rows of x against A_i (or of dy against B_i): the rows come
//           by TMA gather, K is split over a cluster of 1 to 8 CTAs, whose fp32
//           sums meet through distributed shared memory in rank order; v is
//           kept as a sum of bf16 (what a first one leaves goes to a second,
//           and what that leaves to a third)
//   expand  v against B_i (or A_i), 128 x 128 outputs at a time; base comes by
//           TMA gather ahead of use, the sum goes back to its row
//   wgrad   x^T u and dy^T v over an adapter's slots, both operands MN-major
//           as they lie; long adapters in chunks whose parts are added in order
//
// Two choices keep fp32 results fp32.  The tensor cores take bf16, so expand
// multiplies the first two parts of v (2^-16 of v is lost, under a bf16 output
// step of 2^-8) and wgrad all three (24 bits, nothing lost).  And they truncate
// as they accumulate, about 2^-26 of the sum a step, all to one side: 1.6e-5
// of v over 16384 columns.  So no sum stays in tensor memory for more than
// kSegment K-blocks; the epilogue warps add those sums up in registers, rounding
// to nearest.  The extra products and reads hide behind the wide operand.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "lb_common.cuh"
#include "lb_internal.h"
#include "lb_tc.cuh"

namespace lb {
namespace {

using namespace tc;

constexpr int TM = 128;               // slots of a tile
constexpr uint32_t kBox = 64 * 128;   // 64 rows (or slots) of 64 two-byte elements
constexpr int kSegment = 4;           // K-blocks that are summed in tensor memory
constexpr int kParts = 3;             // bf16 that v is the sum of

// ------------------------------------------------------------ the plan
struct Tile {
    int adapter;  // -1: tokens without an adapter
    int rows;     // slots in use, from 1 to TM
};
struct Chunk {  // a run of one adapter's tiles for wgrad
    int adapter, tile0, slots;
    int part;  // where its partial sums go, -1: straight to the gradient
};
struct Multi {  // an adapter of several chunks
    int adapter, part0, parts;
};
struct Plan {
    int *counts;  // tiles, chunks, adapters of several chunks
    Tile *tiles;
    int *perm;  // [tiles][TM]: the token of each slot, `tokens` for none
    Chunk *chunks;
    Multi *multi;
};

struct PlanParams {
    const int32_t *ids;
    int tokens, count;
    int chunk_tiles;  // tiles of a chunk; 0: no chunks wanted
    Plan plan;
    int *status;
};

constexpr int kPlanThreads = 1024, kPlanWarps = 32;

// Exclusive sum over the block of one value per thread; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int *sums, int &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += n;
    }
    __syncthreads();
    if (lane == 31) sums[w] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < kPlanWarps; ++i) {
        const int s = sums[i];
        if (i < w) before += s;
        total += s;
    }
    return before + inc - v;
}

// Each warp takes a run of tokens in order, so that an adapter's tokens keep
// their order and sums over them do not depend on timing.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p)
{
    extern __shared__ int hist[];  // [warp][bin]; bin `count`: no adapter
    __shared__ int sums[kPlanWarps], first_tile[LB_MAX_ADAPTERS + 1];
    const int bins = p.count + 1, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    for (int i = tid; i < kPlanWarps * bins; i += kPlanThreads) hist[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int run = (((p.tokens + kPlanWarps - 1) / kPlanWarps) + 31) & ~31;
    const int t0 = w * run, t1 = min(p.tokens, t0 + run);
    auto bin_of = [&](int t) {
        if (t >= t1) return -1;
        const int id = __ldg(p.ids + t);
        if (id >= p.count) set_status(p.status, LB_ERR_INVALID_ARGUMENT);
        return id < 0 || id >= p.count ? p.count : id;
    };
    int *mine = hist + w * bins;
    for (int t = t0; t < t1; t += 32) {
        const int b = bin_of(t + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, b);
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // per bin: its tokens, and where each warp's share of them begins
    auto total_of = [&](int b) {
        int n = 0;
        for (int i = 0; i < kPlanWarps; ++i) {
            const int k = hist[i * bins + b];
            hist[i * bins + b] = n;
            n += k;
        }
        return n;
    };
    const int n = tid < p.count ? total_of(tid) : 0;
    const int tiles = (n + TM - 1) / TM;
    int all_tiles;
    const int tile0 = block_scan(tiles, sums, all_tiles);
    if (tid < p.count) first_tile[tid] = tile0;
    int none = 0;
    if (tid == 0) {
        none = total_of(p.count);
        first_tile[p.count] = all_tiles;
        p.plan.counts[0] = all_tiles + (none + TM - 1) / TM;
    }
    auto list_tiles = [&](int adapter, int begin, int tokens) {
        for (int i = 0; i * TM < tokens; ++i) p.plan.tiles[begin + i] = Tile{adapter, min(TM, tokens - i * TM)};
        for (int s = tokens; s % TM != 0; ++s) p.plan.perm[begin * TM + s] = p.tokens;
    };
    list_tiles(tid, tile0, n);  // nothing for a thread without a bin
    if (tid == 0) list_tiles(-1, all_tiles, none);
    if (p.chunk_tiles > 0) {  // every adapter has a chunk, so that its gradient is written
        const int parts = tid < p.count ? max(1, (tiles + p.chunk_tiles - 1) / p.chunk_tiles) : 0;
        int all_chunks, all_parts, all_multi;
        const int chunk0 = block_scan(parts, sums, all_chunks);
        const int part0 = block_scan(parts > 1 ? parts : 0, sums, all_parts);
        const int multi = block_scan(parts > 1 ? 1 : 0, sums, all_multi);
        for (int i = 0; i < parts; ++i) {
            const int a = i * p.chunk_tiles;
            const int slots = min(n, (a + p.chunk_tiles) * TM) - a * TM;
            p.plan.chunks[chunk0 + i] = Chunk{tid, tile0 + a, slots, parts > 1 ? part0 + i : -1};
        }
        if (parts > 1) p.plan.multi[multi] = Multi{tid, part0, parts};
        if (tid == 0) {
            p.plan.counts[1] = all_chunks;
            p.plan.counts[2] = all_multi;
        }
    }
    __syncthreads();
    for (int t = t0; t < t1; t += 32) {
        const int b = bin_of(t + lane);
        const uint32_t same = __match_any_sync(0xffffffffu, b);
        int at = 0;
        if (b >= 0) at = mine[b] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (b >= 0) {
            p.plan.perm[first_tile[b] * TM + at] = t + lane;
            if (lane == __ffs(same) - 1) mine[b] += __popc(same);
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------ loads
// Four rows y.x .. y.w of a matrix, 64 columns from x on, to 4 x 128 bytes.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *tm, int x, int4 y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5, %6}], [%7];" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
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
__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ int used_rank(const int32_t *ranks, int rank, int adapter)
{
    return ranks == nullptr ? rank : max(0, min(rank, __ldg(ranks + adapter)));
}

// ------------------------------------------------------------ shrink
// v = s_i W_i x of a tile's rows, W_i [rank x K] (K-major: A_i) or [K x rank]
// (MN-major: B_i).  Grid (splits, tiles, jobs), clusters of `splits` CTAs.
struct ShrinkJob {
    CUtensorMap x, w;
    int k, rank, mn;
    const int32_t *ranks;
    const float *scale;
    uint16_t *v[kParts];  // [slots][rank] each; the third may be null
};
struct ShrinkParams {
    ShrinkJob job[kMaxSiblings];
    Plan plan;
    int *status;
};

constexpr int kShrinkThreads = 192;
constexpr uint32_t kXBytes = TM * 128;  // a K-block of a tile's rows: 64 columns
// two CTAs on an SM: 100 KB each
__host__ __device__ constexpr int shrink_stages(int rank) { return rank > 64 ? 3 : 4; }
__host__ __device__ constexpr uint32_t shrink_w_bytes(int rank) { return rank > 64 ? 2 * kBox : kBox; }
constexpr size_t kShrinkSmem = 1024 + 4 * (kXBytes + kBox) + 128;
constexpr int kMaxRank = LB_MAX_ADAPTER_RANK;
static_assert(4 * (kXBytes + kBox) == 3 * (kXBytes + 2 * kBox), "stages of both widths fill the same memory");
static_assert(TM * (128 + 4) * 4 <= 4 * (kXBytes + kBox), "the sums fit where the stages were");

__global__ void __launch_bounds__(kShrinkThreads, 2) shrink_kernel(const __grid_constant__ ShrinkParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const ShrinkJob &J = p.job[blockIdx.z];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const int stages = shrink_stages(J.rank);
    const uint32_t w_bytes = shrink_w_bytes(J.rank), stage_bytes = kXBytes + w_bytes;
    // full[4], empty[4], acc_full[2], acc_empty[2], drain, the tmem address
    const uint32_t bars = base + 4 * (kXBytes + kBox);
    const uint32_t full0 = bars, empty0 = bars + 32, accf0 = bars + 64, acce0 = bars + 80, drain = bars + 96;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem_raw + (drain + 8 - raw));
    __shared__ int abort_shared;
    volatile int &abort_flag = abort_shared;
    const int splits = gridDim.x, split = blockIdx.x, tile = blockIdx.y;

    if (warp == 1) {
        if (lane == 0) {
            for (int s = 0; s < stages; ++s) {
                mbar_init(full0 + 8 * s, 1);
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
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const bool in_plan = tile < p.plan.counts[0];
    const Tile T = in_plan ? p.plan.tiles[tile] : Tile{-1, 0};
    const int rank = T.adapter >= 0 ? used_rank(J.ranks, J.rank, T.adapter) : 0;
    const bool live = rank > 0;  // uniform over the cluster
    const int nr = (J.rank + 15) & ~15;
    const int nkb = (J.k + 63) / 64, kb0 = (int)((int64_t)nkb * split / splits), kb1 = (int)((int64_t)nkb * (split + 1) / splits);
    if (live && warp == 0) {
        // TMA: lane q brings rows 4q .. 4q + 3 (rows past the tile's stay as
        // they were: they end in rows of v that are written as zeros)
        const int quads = (T.rows + 3) >> 2;
        const int4 rows = *reinterpret_cast<const int4 *>(p.plan.perm + tile * TM + 4 * lane);
        const int boxes = J.mn ? (J.rank + 63) / 64 : 1;
        const uint32_t tx = (uint32_t)quads * 512u + (J.mn ? (uint32_t)boxes * kBox : (uint32_t)nr * 128u);
        int g = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
            const int s = g % stages;
            const uint32_t ph = (uint32_t)(g / stages) & 1u;
            const bool ok = mbar_wait(empty0 + 8 * s, ph ^ 1u) && !abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            const uint32_t sx = base + s * stage_bytes, sw = sx + kXBytes, bar = full0 + 8 * s;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, tx);
                if (J.mn)
                    for (int b = 0; b < boxes; ++b) tma_load_3d(sw + b * kBox, &J.w, 64 * b, 64 * kb, T.adapter, bar);
                else
                    tma_load_3d(sw, &J.w, 64 * kb, 0, T.adapter, bar);
            }
            __syncwarp();
            if (lane < quads) tma_gather4(sx + lane * 512u, &J.x, 64 * kb, rows, bar);
        }
        if (abort_flag && lane == 0)
            for (int q = (g > stages ? g - stages : 0); q < g; ++q)
                mbar_wait(full0 + 8 * (q % stages), (uint32_t)(q / stages) & 1u);
    } else if (live && warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_of(nr, false, J.mn != 0);
            int g = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int s = g % stages, seg = g / kSegment, b = seg & 1;
                const bool first = g % kSegment == 0;
                if ((first && !mbar_wait(acce0 + 8 * b, ((uint32_t)(seg >> 1) & 1u) ^ 1u)) ||
                    !mbar_wait(full0 + 8 * s, (uint32_t)(g / stages) & 1u) || abort_flag) {
                    abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t sx = base + s * stage_bytes, sw = sx + kXBytes;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t bd = J.mn ? smem_desc_mn(sw + 2048u * kk) : smem_desc(sw + 32u * kk);
                    umma(tmem + 128 * b, smem_desc(sx + 32u * kk), bd, idesc, !first || kk != 0 ? 1u : 0u);
                }
                umma_commit(empty0 + 8 * s);
                if (g % kSegment == kSegment - 1 || kb + 1 == kb1) umma_commit(accf0 + 8 * b);
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else if (live) {
        // this CTA's sums, a row a lane: the segments in registers, then to
        // shared memory where the stages were (the last segment's MMAs, and
        // with them every copy, are done by then)
        const int quad = warp & 3, row = 32 * quad + lane;
        float sum[kMaxRank];
#pragma unroll
        for (int c = 0; c < kMaxRank; ++c) sum[c] = 0.0f;
        const int segs = (kb1 - kb0 + kSegment - 1) / kSegment;
        bool ok = true;
        for (int seg = 0; seg < segs; ++seg) {
            const int b = seg & 1;
            ok = !abort_flag && mbar_wait(accf0 + 8 * b, (uint32_t)(seg >> 1) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                abort_flag = 1;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kMaxRank; c += 16) {
                if (c < nr) {
                    uint32_t v[16];
                    tmem_ld16(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * b + c), v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce0 + 8 * b);
        }
        if (ok) {
#pragma unroll
            for (int c = 0; c < kMaxRank; c += 4)
                if (c < nr)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + (uint32_t)(row * (nr + 4) + c) * 4u),
                                 "r"(__float_as_uint(sum[c])), "r"(__float_as_uint(sum[c + 1])),
                                 "r"(__float_as_uint(sum[c + 2])), "r"(__float_as_uint(sum[c + 3]))
                                 : "memory");
        }
    }
    __syncthreads();
    if (splits > 1) cluster_sync();
    if (live) {
        // rows 128 split / splits .. of the tile: every CTA's sums in rank order
        const int per = TM / splits, r0 = split * per, cols4 = J.rank / 4;
        const float scale = J.scale != nullptr ? __ldg(J.scale + T.adapter) : 1.0f;
        for (int i = threadIdx.x; i < per * cols4; i += kShrinkThreads) {
            const int row = r0 + i / cols4, c = 4 * (i % cols4);
            const uint32_t at = base + (uint32_t)(row * (nr + 4) + c) * 4u;
            float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row < T.rows) {
                for (int q = 0; q < splits; ++q) {
                    const float4 v = ld_shared_cluster_f4(splits > 1 ? map_shared_addr(at, (uint32_t)q) : at);
                    f[0] += v.x, f[1] += v.y, f[2] += v.z, f[3] += v.w;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = row < T.rows && c + e < rank ? f[e] * scale : 0.0f;
            const int64_t o = ((int64_t)tile * TM + row) * J.rank + c;
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                if (J.v[q] == nullptr) break;
                const uint2 part = make_uint2(pack_bf162(f[0], f[1]), pack_bf162(f[2], f[3]));
                *reinterpret_cast<uint2 *>(J.v[q] + o) = part;
                const float h[4] = {__uint_as_float(part.x << 16), __uint_as_float(part.x & 0xffff0000u),
                                    __uint_as_float(part.y << 16), __uint_as_float(part.y & 0xffff0000u)};
                // what is left (exact); an infinity or NaN is all in the first
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = fabsf(h[e]) < __int_as_float(0x7f800000) ? f[e] - h[e] : 0.0f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (splits > 1) cluster_sync();  // the others may still read this CTA's sums
    if (abort_flag && threadIdx.x == 0) set_status(p.status, LB_ERR_DEVICE_TIMEOUT);
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ------------------------------------------------------------ expand
// y = base + W_i v of every tile, 128 columns a unit.  W_i [n x rank]
// (K-major: B_i) or [rank x n] (MN-major: A_i).  Persistent CTAs, each with a
// run of consecutive units (chunk fastest, so a tile's v stays).
struct ExpandJob {
    CUtensorMap base, w, hi, lo;
    int n, rank, mn, chunks;
    const int32_t *ranks;
    uint16_t *y;
    int64_t ldy;
    int in_place;
};
struct ExpandParams {
    ExpandJob job[kMaxSiblings];
    int njobs, per_tile;  // chunks of all jobs
    int tokens;
    Plan plan;
    int *status;
};

constexpr int kExpandWarps = 8;  // of the epilogue
constexpr int kExpandThreads = 64 + 32 * kExpandWarps;
constexpr uint32_t kBaseBytes = TM * 256;  // 128 columns of a tile's rows: two halves of 64
constexpr uint32_t kVBytes = TM * 128;     // 64 columns of hi or lo
// NK: 64-wide blocks of the rank
template <int NK>
struct Expand {
    static constexpr int kStages = NK == 1 ? 3 : 2;
    static constexpr int kVBufs = NK == 1 ? 2 : 1;
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
                mbar_init(full0 + 8 * s, 1);
                mbar_init(empty0 + 8 * s, kExpandWarps);
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
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int64_t units = (int64_t)p.plan.counts[0] * p.per_tile;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    // every role walks the same units; `kind`: 0 nothing to do, 1 copy base, 2 add
    struct Unit {
        int tile, job, chunk, kind;
        Tile t;
        bool fresh;  // first unit of its tile and job here: v is loaded
    };
    int last_tile = -1, last_job = -1, tile_kind = 0;
    Tile tile_info{-1, 0};
    auto next = [&](int64_t u) {
        Unit q;
        q.tile = (int)(u / p.per_tile);
        int c = (int)(u - (int64_t)q.tile * p.per_tile);
        q.job = 0;
        while (c >= p.job[q.job].chunks) c -= p.job[q.job++].chunks;
        q.chunk = c;
        q.fresh = q.tile != last_tile || q.job != last_job;
        if (q.fresh) {
            last_tile = q.tile;
            last_job = q.job;
            tile_info = p.plan.tiles[q.tile];
            const ExpandJob &J = p.job[q.job];
            const int r = tile_info.adapter >= 0 ? used_rank(J.ranks, J.rank, tile_info.adapter) : 0;
            tile_kind = r > 0 ? 2 : J.in_place ? 0 : 1;
        }
        q.kind = tile_kind;
        q.t = tile_info;
        q.fresh = q.fresh && tile_kind == 2;
        return q;
    };

    if (warp == 0) {
        int g = 0, nv = 0;
        int4 rows = make_int4(0, 0, 0, 0);
        int rows_tile = -1;
        for (int64_t u = u0; u < u1; ++u) {
            const Unit q = next(u);
            if (q.kind == 0) continue;
            const ExpandJob &J = p.job[q.job];
            if (rows_tile != q.tile) {
                rows = *reinterpret_cast<const int4 *>(p.plan.perm + q.tile * TM + 4 * lane);
                rows_tile = q.tile;
            }
            bool ok = true;
            if (q.fresh) {
                const int b = nv % S::kVBufs;
                ok = mbar_wait(vempty0 + 8 * b, ((uint32_t)(nv / S::kVBufs) & 1u) ^ 1u) && !abort_flag;
                if (ok && lane == 0) {
                    const uint32_t bar = vfull0 + 8 * b, dst = sV + b * S::kV;
                    mbar_arrive_expect_tx(bar, S::kV);
                    for (int k = 0; k < NK; ++k) {
                        tma_load_2d(dst + (2 * k) * kVBytes, &J.hi, 64 * k, q.tile * TM, bar);
                        tma_load_2d(dst + (2 * k + 1) * kVBytes, &J.lo, 64 * k, q.tile * TM, bar);
                    }
                }
                ++nv;
            }
            const int s = g % S::kStages;
            ok = ok && mbar_wait(empty0 + 8 * s, ((uint32_t)(g / S::kStages) & 1u) ^ 1u) && !abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            const int quads = (q.t.rows + 3) >> 2, c0 = 128 * q.chunk;
            const uint32_t dst = sS + s * S::kStage, bar = full0 + 8 * s;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, (uint32_t)quads * 1024u + (q.kind == 2 ? S::kW : 0u));
                if (q.kind == 2) {
                    for (int k = 0; k < NK; ++k) {
                        if (J.mn) {  // 64 rows of the rank x 128 columns
                            tma_load_3d(dst + (2 * k) * kBox, &J.w, c0, 64 * k, q.t.adapter, bar);
                            tma_load_3d(dst + (2 * k + 1) * kBox, &J.w, c0 + 64, 64 * k, q.t.adapter, bar);
                        } else {  // 128 rows x 64 columns of the rank
                            tma_load_3d(dst + k * 2 * kBox, &J.w, 64 * k, c0, q.t.adapter, bar);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane < quads) {
                tma_gather4(dst + S::kW + lane * 512u, &J.base, c0, rows, bar);
                tma_gather4(dst + S::kW + kBaseBytes / 2 + lane * 512u, &J.base, c0 + 64, rows, bar);
            }
            ++g;
        }
        if (abort_flag && lane == 0) {
            for (int i = (g > S::kStages ? g - S::kStages : 0); i < g; ++i)
                mbar_wait(full0 + 8 * (i % S::kStages), (uint32_t)(i / S::kStages) & 1u);
            for (int i = (nv > S::kVBufs ? nv - S::kVBufs : 0); i < nv; ++i)
                mbar_wait(vfull0 + 8 * (i % S::kVBufs), (uint32_t)(i / S::kVBufs) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int g = 0, nv = 0, na = 0;
            for (int64_t u = u0; u < u1 && !abort_flag; ++u) {
                const Unit q = next(u);
                if (q.kind == 0) continue;
                const ExpandJob &J = p.job[q.job];
                const int s = g % S::kStages, ab = na & 1;
                if (q.kind == 1) {  // no product; but no phase of a stage is skipped
                    if (!mbar_wait(full0 + 8 * s, (uint32_t)(g / S::kStages) & 1u)) {
                        abort_flag = 1;
                        break;
                    }
                    ++g;
                    continue;
                }
                if (q.fresh) {
                    if (nv > 0) umma_commit(vempty0 + 8 * ((nv - 1) % S::kVBufs));  // the tile before is read
                    const int b = nv % S::kVBufs;
                    if (!mbar_wait(vfull0 + 8 * b, (uint32_t)(nv / S::kVBufs) & 1u)) {
                        abort_flag = 1;
                        break;
                    }
                    ++nv;
                }
                if (!mbar_wait(acce0 + 8 * ab, ((uint32_t)(na >> 1) & 1u) ^ 1u) ||
                    !mbar_wait(full0 + 8 * s, (uint32_t)(g / S::kStages) & 1u) || abort_flag) {
                    abort_flag = 1;
                    break;
                }
                tc_fence_after();
                const uint32_t v = sV + ((nv - 1) % S::kVBufs) * S::kV, w = sS + s * S::kStage, acc = tmem + 128 * ab;
                const uint32_t idesc = idesc_of(128, false, J.mn != 0);
                const int steps = (J.rank + 15) / 16;
                for (int i = 0; i < steps; ++i) {
                    const int k = i >> 2, kk = i & 3;
                    const uint64_t bd = J.mn ? smem_desc_mn(w + k * 2 * kBox + 2048u * kk) : smem_desc(w + k * 2 * kBox + 32u * kk);
                    umma(acc, smem_desc(v + (2 * k) * kVBytes + 32u * kk), bd, idesc, i != 0 ? 1u : 0u);
                    umma(acc, smem_desc(v + (2 * k + 1) * kVBytes + 32u * kk), bd, idesc, 1u);
                }
                umma_commit(accf0 + 8 * ab);
                ++g;
                ++na;
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else {
        // epilogue: warp e takes rows 32 (warp % 4) .. and 64 of the unit's columns
        const int quad = warp & 3, half = (warp - 2) >> 2, row = 32 * quad + lane;
        int g = 0, na = 0, tok = 0, tok_tile = -1;
        for (int64_t u = u0; u < u1; ++u) {
            const Unit q = next(u);
            if (q.kind == 0) continue;
            const ExpandJob &J = p.job[q.job];
            if (tok_tile != q.tile) {
                tok = p.plan.perm[q.tile * TM + row];
                tok_tile = q.tile;
            }
            const int s = g % S::kStages, ab = na & 1;
            bool ok = !abort_flag && mbar_wait(full0 + 8 * s, (uint32_t)(g / S::kStages) & 1u);
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
                    uint32_t v[32];
                    tmem_ld32(tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(128 * ab + 64 * half + 32 * h), v);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t a = at + (uint32_t)(((4 * h + c) ^ (row & 7)) << 4);
                        uint32_t b[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                                     : "r"(a)
                                     : "memory");
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float f0 = __uint_as_float(b[e] << 16) + __uint_as_float(v[8 * c + 2 * e]);
                            const float f1 = __uint_as_float(b[e] & 0xffff0000u) + __uint_as_float(v[8 * c + 2 * e + 1]);
                            b[e] = pack_bf162(f0, f1);
                        }
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(b[0]), "r"(b[1]), "r"(b[2]),
                                     "r"(b[3])
                                     : "memory");
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * ab);
                ++na;
            }
            // back to the rows of y: 8 lanes a row, 128 bytes
            const int col = 128 * q.chunk + 64 * half + 8 * (lane & 7);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3);  // within this warp's 32 rows
                const int t = __shfl_sync(0xffffffffu, tok, r);
                if (t < p.tokens && col < J.n) {
                    uint4 o;
                    const int tr = 32 * quad + r;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                                 : "r"(tile + (uint32_t)tr * 128u + (uint32_t)(((lane & 7) ^ (tr & 7)) << 4))
                                 : "memory");
                    *reinterpret_cast<uint4 *>(J.y + (int64_t)t * J.ldy + col) = o;
                }
            }
            fence_async_shared();  // the next copy into this stage comes after these accesses
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * s);
            ++g;
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

// ------------------------------------------------------------ wgrad
// dA_i[r][n] = sum over an adapter's slots of u[slot][r] x[slot][n], and dB_i
// the same of v and dy with the result [n][r]: D[n][r], 128 columns n a unit,
// the slots as K; both operands MN-major (slots outermost).
struct WgradJob {
    CUtensorMap x, v[kParts];
    int n, tiles;      // columns, 128-wide units of them
    int transposed;    // the gradient is [r][n]
    float *out;        // [adapter][...]
    int64_t part_off;  // within a part
};
struct AdapterWgradParams {
    WgradJob job[2];
    int rank;
    const int32_t *ranks;
    Plan plan;
    float *part;         // [part][part_size]
    int64_t part_size;
    int *status;
};

constexpr int kWgradThreads = 192;
template <int NK>
struct WgradShape {
    static constexpr int kStages = NK == 1 ? 5 : 3;
    static constexpr uint32_t kStage = 2 * kBox + kParts * NK * kBox;
    static constexpr size_t kSmem = 1024 + kStages * kStage + 256;
};

template <int NK>
__global__ void __launch_bounds__(kWgradThreads, 1) adapter_wgrad_kernel(const __grid_constant__ AdapterWgradParams p)
{
    using S = WgradShape<NK>;
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
                mbar_init(full0 + 8 * s, 1);
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
        tmem_alloc(smem_u32(tmem_slot), 512);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const int per = p.job[0].tiles + p.job[1].tiles;
    const int64_t units = (int64_t)p.plan.counts[1] * per;
    const int nr = (p.rank + 15) & ~15;
    struct Unit {
        Chunk c;
        int job, n0, nkb;
    };
    auto unit_of = [&](int64_t u) {
        Unit q;
        q.c = p.plan.chunks[u / per];
        const int m = (int)(u % per);
        q.job = m >= p.job[0].tiles;
        q.n0 = 128 * (q.job ? m - p.job[0].tiles : m);
        q.nkb = (q.c.slots + 63) / 64;
        if (used_rank(p.ranks, p.rank, q.c.adapter) == 0) q.nkb = 0;
        return q;
    };

    if (warp == 0) {
        // lanes 0 .. 15 bring the 64 slots' rows of columns n0 .., lanes 16 .. 31 of n0 + 64 ..
        int g = 0;
        bool stop = false;
        for (int64_t u = blockIdx.x; u < units && !stop; u += gridDim.x) {
            const Unit q = unit_of(u);
            const WgradJob &J = p.job[q.job];
            const int *perm = p.plan.perm + q.c.tile0 * TM + 4 * (lane & 15);
            int4 rows = make_int4(0, 0, 0, 0);
            if (q.nkb > 0) rows = *reinterpret_cast<const int4 *>(perm);
            for (int kb = 0; kb < q.nkb; ++kb, ++g) {
                const int s = g % S::kStages;
                const int4 now = rows;
                if (kb + 1 < q.nkb) rows = *reinterpret_cast<const int4 *>(perm + 64 * (kb + 1));
                const bool ok = mbar_wait(empty0 + 8 * s, ((uint32_t)(g / S::kStages) & 1u) ^ 1u) && !abort_flag;
                if (!__all_sync(0xffffffffu, ok)) {
                    abort_flag = 1;
                    stop = true;
                    break;
                }
                const uint32_t dst = base + s * S::kStage, bar = full0 + 8 * s;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, S::kStage);
                    const int slot = q.c.tile0 * TM + 64 * kb;
                    for (int i = 0; i < kParts; ++i)
                        for (int k = 0; k < NK; ++k) tma_load_2d(dst + (2 + i * NK + k) * kBox, &J.v[i], 64 * k, slot, bar);
                }
                __syncwarp();
                tma_gather4(dst + (lane >> 4) * kBox + (lane & 15) * 512u, &J.x, q.n0 + 64 * (lane >> 4), now, bar);
            }
        }
        if (abort_flag && lane == 0)
            for (int i = (g > S::kStages ? g - S::kStages : 0); i < g; ++i)
                mbar_wait(full0 + 8 * (i % S::kStages), (uint32_t)(i / S::kStages) & 1u);
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = idesc_of(nr, true, true);
            int g = 0, na = 0;  // K-blocks and segments so far
            for (int64_t u = blockIdx.x; u < units && !abort_flag; u += gridDim.x) {
                const Unit q = unit_of(u);
                for (int kb = 0; kb < q.nkb; ++kb, ++g) {
                    const int s = g % S::kStages, ab = na & 1;
                    const bool first = kb % kSegment == 0;
                    if ((first && !mbar_wait(acce0 + 8 * ab, ((uint32_t)(na >> 1) & 1u) ^ 1u)) ||
                        !mbar_wait(full0 + 8 * s, (uint32_t)(g / S::kStages) & 1u) || abort_flag) {
                        abort_flag = 1;
                        break;
                    }
                    tc_fence_after();
                    // the first part of v in one sum, the smaller ones in another
                    const uint32_t a = base + s * S::kStage, b = a + 2 * kBox, acc = tmem + 256 * ab;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ad = smem_desc_mn(a + 2048u * kk);
                        const uint32_t more = !first || kk != 0 ? 1u : 0u;
                        umma(acc, ad, smem_desc_mn(b + 2048u * kk), idesc, more);
#pragma unroll
                        for (int i = 1; i < kParts; ++i)
                            umma(acc + 128, ad, smem_desc_mn(b + i * NK * kBox + 2048u * kk), idesc, i > 1 ? 1u : more);
                    }
                    umma_commit(empty0 + 8 * s);
                    if (kb % kSegment == kSegment - 1 || kb + 1 == q.nkb) {
                        umma_commit(accf0 + 8 * ab);
                        ++na;
                    }
                }
            }
            umma_commit(drain);
            if (!mbar_wait(drain, 0)) abort_flag = 1;
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;
        int na = 0;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
            const Unit q = unit_of(u);
            const WgradJob &J = p.job[q.job];
            const int used = used_rank(p.ranks, p.rank, q.c.adapter);
            float sum[64 * NK];
#pragma unroll
            for (int c = 0; c < 64 * NK; ++c) sum[c] = 0.0f;
            bool ok = !abort_flag;
            for (int kb = 0; kb < q.nkb; kb += kSegment, ++na) {
                const int ab = na & 1;
                ok = !abort_flag && mbar_wait(accf0 + 8 * ab, (uint32_t)(na >> 1) & 1u);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 64 * NK; c += 16) {
                    if (c < nr) {
                        uint32_t v[16], w[16];
                        const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(256 * ab + c);
                        tmem_ld16(at, v);
                        tmem_ld16(at + 128, w);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[c + i] += __uint_as_float(v[i]) + __uint_as_float(w[i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce0 + 8 * ab);
            }
            if (!__all_sync(0xffffffffu, ok)) {
                abort_flag = 1;
                break;
            }
            const int n = q.n0 + 32 * quad + lane;
            float *out = q.c.part >= 0 ? p.part + q.c.part * p.part_size + J.part_off
                                       : J.out + (int64_t)q.c.adapter * p.rank * J.n;
            if (n >= J.n) continue;
            if (J.transposed) {
#pragma unroll
                for (int c = 0; c < 64 * NK; ++c)
                    if (c < p.rank) out[(int64_t)c * J.n + n] = c < used ? sum[c] : 0.0f;
            } else {
#pragma unroll
                for (int c = 0; c < 64 * NK; c += 4)
                    if (c < p.rank)
                        *reinterpret_cast<float4 *>(out + (int64_t)n * p.rank + c) =
                            make_float4(c < used ? sum[c] : 0.0f, c + 1 < used ? sum[c + 1] : 0.0f,
                                        c + 2 < used ? sum[c + 2] : 0.0f, c + 3 < used ? sum[c + 3] : 0.0f);
            }
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

// The gradients of adapters of several chunks: their parts, added in order.
struct SumParams {
    Plan plan;
    const float *part;
    int64_t part_size, a_size, b_size;  // floats
    float *da, *db;
};
__global__ void __launch_bounds__(256) sum_parts_kernel(const SumParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const int multi = p.plan.counts[2];
    const int64_t quads = p.part_size / 4;
    for (int m = 0; m < multi; ++m) {
        const Multi e = p.plan.multi[m];
        const float4 *src = reinterpret_cast<const float4 *>(p.part + e.part0 * p.part_size);
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < quads; i += (int64_t)gridDim.x * blockDim.x) {
            float4 s = src[i];
            for (int q = 1; q < e.parts; ++q) {
                const float4 v = src[q * quads + i];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            float *dst = 4 * i < p.a_size ? p.da + e.adapter * p.a_size + 4 * i : p.db + e.adapter * p.b_size + (4 * i - p.a_size);
            *reinterpret_cast<float4 *>(dst) = s;
        }
    }
}

// ------------------------------------------------------------ host side
size_t align256(size_t b) { return (b + 255) & ~size_t(255); }

// Tiles of a batch: at most one partial tile per adapter in use, and for the
// tokens without one.
int most_tiles(int tokens, int count) { return tokens / TM + std::min(count + 1, tokens); }

struct Layout {
    size_t counts, tiles, perm, chunks, multi, v[kMaxSiblings][kParts], part, total;
};
Layout layout_of(int tokens, int count, int nv, const int *ranks, int parts, int max_chunks, size_t part_floats)
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
    L.chunks = take((size_t)max_chunks * sizeof(Chunk));
    L.multi = take((size_t)max_chunks * sizeof(Multi));
    for (int j = 0; j < nv; ++j)
        for (int q = 0; q < parts; ++q) L.v[j][q] = take(tiles * TM * (size_t)ranks[j] * 2);
    L.part = take(part_floats * sizeof(float));
    L.total = off;
    return L;
}

Plan plan_at(const Layout &L, uint8_t *ws)
{
    Plan p;
    p.counts = reinterpret_cast<int *>(ws + L.counts);
    p.tiles = reinterpret_cast<Tile *>(ws + L.tiles);
    p.perm = reinterpret_cast<int *>(ws + L.perm);
    p.chunks = reinterpret_cast<Chunk *>(ws + L.chunks);
    p.multi = reinterpret_cast<Multi *>(ws + L.multi);
    return p;
}

// Rows of a bf16 matrix, gathered four at a time, 64 columns wide.
cudaError_t encode_gather(CUtensorMap *tm, const void *ptr, int rows, int cols, int64_t ld)
{
    return encode_2d(tm, ptr, rows, cols, ld, true, 1);
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
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, int cluster, const P &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_plan(const int32_t *ids, int tokens, int count, int chunk_tiles, const Plan &plan, const DeviceInfo &dev,
                        cudaStream_t stream)
{
    const PlanParams p{ids, tokens, count, chunk_tiles, plan, dev.status};
    return launch(plan_kernel, dim3(1), kPlanThreads, sizeof(int) * kPlanWarps * (size_t)(count + 1), 1, p, stream);
}

// CTAs a tile's K is split over: as few as give every SM its two CTAs, with at
// least four K-blocks each.
int shrink_splits(int tokens, int jobs, int k, int sms)
{
    const int tiles = (tokens + TM - 1) / TM * jobs, nkb = (k + 63) / 64;
    int s = 1;
    while (s < 8 && tiles * s * 2 <= 2 * sms && nkb >= 8 * s) s *= 2;
    return s;
}

cudaError_t launch_expand(const ExpandParams &p, int rank, const DeviceInfo &dev, cudaStream_t stream)
{
    const dim3 grid((unsigned)dev.sm_count);
    return rank <= 64 ? launch(expand_kernel<1>, grid, kExpandThreads, Expand<1>::kSmem, 1, p, stream)
                      : launch(expand_kernel<2>, grid, kExpandThreads, Expand<2>::kSmem, 1, p, stream);
}

// Tiles of a wgrad chunk, for about three units an SM when one adapter has all tokens.
int wgrad_chunk_tiles(int tokens, int n_in, int n_out, int sms)
{
    const int tiles = (tokens + TM - 1) / TM, per = (n_in + 127) / 128 + (n_out + 127) / 128;
    const int chunks = std::max(1, std::min(tiles, (3 * sms + per - 1) / per));
    return (tiles + chunks - 1) / chunks;
}
// Parts: an adapter of several chunks has more than chunk_tiles tiles of
// tokens, so all of them have fewer than 2 tokens / (128 chunk_tiles) chunks.
int wgrad_parts(int tokens, int chunk_tiles) { return chunk_tiles * TM >= tokens ? 0 : 2 * tokens / (TM * chunk_tiles) + 1; }

constexpr int kSmsForPlan = 148;  // plans are made for this many SMs, so that workspaces do not depend on the device

}  // namespace

cudaError_t adapters_mma_prepare_device(const DeviceInfo &dev)
{
    (void)dev;
    cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(int) * kPlanWarps * (LB_MAX_ADAPTERS + 1)));
    auto allow = [&](auto kernel, size_t bytes) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    };
    allow(shrink_kernel, kShrinkSmem);
    allow(expand_kernel<1>, Expand<1>::kSmem);
    allow(expand_kernel<2>, Expand<2>::kSmem);
    allow(adapter_wgrad_kernel<1>, WgradShape<1>::kSmem);
    allow(adapter_wgrad_kernel<2>, WgradShape<2>::kSmem);
    return e;
}

size_t adapters_mma_workspace_bytes(int tokens, int count, int nproj, const int *ranks)
{
    return layout_of(tokens, count, nproj, ranks, 2, 0, 0).total;
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
    const Layout L = layout_of(a.tokens, a.count, a.nproj, ranks, 2, 0, 0);
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const Plan plan = plan_at(L, ws);
    const int tiles = most_tiles(a.tokens, a.count);
    ShrinkParams sp{};
    ExpandParams ep{};
    sp.plan = ep.plan = plan;
    sp.status = ep.status = dev.status;
    ep.njobs = a.nproj;
    ep.tokens = a.tokens;
    CUtensorMap mx;
    e = encode_gather(&mx, a.x, a.tokens, a.n_in, a.ldx);
    for (int j = 0; j < a.nproj && e == cudaSuccess; ++j) {
        const AdapterProj &P = a.proj[j];
        ShrinkJob &s = sp.job[j];
        s.x = mx;
        s.k = a.n_in;
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
        x.y = P.y;
        x.ldy = P.ldy;
        x.in_place = P.base == P.y;
        if (e == cudaSuccess) e = encode_gather(&x.base, P.base, a.tokens, P.n_out, P.ldbase);
        if (e == cudaSuccess) e = encode_3d(&x.w, P.b, P.rank, P.n_out, a.count, 128);
        if (e == cudaSuccess) e = encode_2d(&x.hi, s.v[0], tiles * TM, P.rank, P.rank, true, TM);
        if (e == cudaSuccess) e = encode_2d(&x.lo, s.v[1], tiles * TM, P.rank, P.rank, true, TM);
    }
    if (e == cudaSuccess) e = launch_plan(a.ids, a.tokens, a.count, 0, plan, dev, stream);
    const int splits = shrink_splits(a.tokens, a.nproj, a.n_in, dev.sm_count);
    if (e == cudaSuccess)
        e = launch(shrink_kernel, dim3((unsigned)splits, (unsigned)tiles, (unsigned)a.nproj), kShrinkThreads, kShrinkSmem,
                   splits, sp, stream);
    if (e == cudaSuccess) e = launch_expand(ep, widest, dev, stream);
    return e;
}

size_t adapters_mma_backward_workspace_bytes(int tokens, int n_in, int n_out, int count, int rank)
{
    const int ct = wgrad_chunk_tiles(tokens, n_in, n_out, kSmsForPlan), parts = wgrad_parts(tokens, ct);
    const int ranks[2] = {rank, rank};
    return layout_of(tokens, count, 2, ranks, kParts, count + parts,
                     (size_t)parts * (size_t)rank * ((size_t)n_in + (size_t)n_out)).total;
}

cudaError_t adapters_mma_backward(const AdaptersBwdArgs &b, const DeviceInfo &dev, cudaStream_t stream)
{
    cudaError_t e = get_encoder();
    if (e != cudaSuccess) return e;
    const int ct = wgrad_chunk_tiles(b.tokens, b.n_in, b.n_out, kSmsForPlan), parts = wgrad_parts(b.tokens, ct);
    const int ranks[2] = {b.rank, b.rank};
    const int64_t a_size = (int64_t)b.rank * b.n_in, b_size = (int64_t)b.rank * b.n_out;
    const Layout L = layout_of(b.tokens, b.count, 2, ranks, kParts, b.count + parts, (size_t)parts * (size_t)(a_size + b_size));
    uint8_t *ws = static_cast<uint8_t *>(b.workspace);
    const Plan plan = plan_at(L, ws);
    const int tiles = most_tiles(b.tokens, b.count);
    uint16_t *v[2][kParts];  // v, then u
    CUtensorMap mx, mdy, mhi, mlo;
    for (int q = 0; q < 2; ++q)
        for (int i = 0; i < kParts; ++i) v[q][i] = reinterpret_cast<uint16_t *>(ws + L.v[q][i]);
    e = encode_2d(&mhi, v[1][0], tiles * TM, b.rank, b.rank, true, TM);
    if (e == cudaSuccess) e = encode_2d(&mlo, v[1][1], tiles * TM, b.rank, b.rank, true, TM);
    if (e == cudaSuccess) e = encode_gather(&mx, b.x, b.tokens, b.n_in, b.ldx);
    if (e == cudaSuccess) e = encode_gather(&mdy, b.dy, b.tokens, b.n_out, b.lddy);
    ShrinkParams sp{};
    sp.plan = plan;
    sp.status = dev.status;
    for (int q = 0; q < 2; ++q) {
        ShrinkJob &s = sp.job[q];
        s.x = q ? mdy : mx;
        s.k = q ? b.n_out : b.n_in;
        s.rank = b.rank;
        s.mn = q;
        s.ranks = b.ranks;
        s.scale = b.scale;
        for (int i = 0; i < kParts; ++i) s.v[i] = v[q][i];
    }
    if (e == cudaSuccess) e = encode_3d(&sp.job[0].w, b.a, b.n_in, b.rank, b.count, (b.rank + 15) & ~15);
    if (e == cudaSuccess) e = encode_3d(&sp.job[1].w, b.b, b.rank, b.n_out, b.count, 64);
    if (e == cudaSuccess) e = launch_plan(b.ids, b.tokens, b.count, ct, plan, dev, stream);
    const int splits = shrink_splits(b.tokens, 2, std::min(b.n_in, b.n_out), dev.sm_count);
    if (e == cudaSuccess)
        e = launch(shrink_kernel, dim3((unsigned)splits, (unsigned)tiles, 2), kShrinkThreads, kShrinkSmem, splits, sp, stream);
    if (b.dx != nullptr && e == cudaSuccess) {
        ExpandParams ep{};
        ep.plan = plan;
        ep.status = dev.status;
        ep.njobs = 1;
        ep.tokens = b.tokens;
        ExpandJob &x = ep.job[0];
        x.n = b.n_in;
        x.rank = b.rank;
        x.mn = 1;
        x.chunks = ep.per_tile = (b.n_in + 127) / 128;
        x.ranks = b.ranks;
        x.y = b.dx;
        x.ldy = b.lddx;
        x.in_place = b.dx_base == b.dx;
        x.hi = mhi;
        x.lo = mlo;
        e = encode_gather(&x.base, b.dx_base, b.tokens, b.n_in, b.lddxbase);
        if (e == cudaSuccess) e = encode_3d(&x.w, b.a, b.n_in, b.rank, b.count, 64);
        if (e == cudaSuccess) e = launch_expand(ep, b.rank, dev, stream);
    }
    if (e != cudaSuccess) return e;
    AdapterWgradParams wp{};
    wp.rank = b.rank;
    wp.ranks = b.ranks;
    wp.plan = plan;
    wp.part = reinterpret_cast<float *>(ws + L.part);
    wp.part_size = a_size + b_size;
    wp.status = dev.status;
    for (int q = 0; q < 2; ++q) {  // dA from x and u, dB from dy and v
        WgradJob &w = wp.job[q];
        w.x = q ? mdy : mx;
        for (int i = 0; i < kParts && e == cudaSuccess; ++i)
            e = encode_2d(&w.v[i], v[1 - q][i], tiles * TM, b.rank, b.rank, true, 64);
        w.n = q ? b.n_out : b.n_in;
        w.tiles = (w.n + 127) / 128;
        w.transposed = !q;
        w.out = q ? b.db : b.da;
        w.part_off = q ? a_size : 0;
    }
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)dev.sm_count);
    e = b.rank <= 64 ? launch(adapter_wgrad_kernel<1>, grid, kWgradThreads, WgradShape<1>::kSmem, 1, wp, stream)
                     : launch(adapter_wgrad_kernel<2>, grid, kWgradThreads, WgradShape<2>::kSmem, 1, wp, stream);
    if (e != cudaSuccess || parts == 0) return e;
    const SumParams qp{plan, wp.part, wp.part_size, a_size, b_size, b.da, b.db};
    return launch(sum_parts_kernel, dim3((unsigned)(2 * dev.sm_count)), 256, 0, 1, qp, stream);
}

}  // namespace lb
