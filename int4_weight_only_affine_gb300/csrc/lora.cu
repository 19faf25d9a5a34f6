// f16_lora: low-rank adapters of many requests beside a shared projection,
//     out[m] = y[m] + s_a (x[m] A_a^T) B_a^T,   a = ids[m]  (negative: out = y).
// The columns may be cut into slices (q | k | v, gate | up) with an A each: B's
// rows of a slice multiply that slice's h = x A^T.
//
// What bounds it: y is read and out written once, x read once, each adapter in
// use read once; the products (2 r flops an element of x and of y) are small
// beside that up to ranks of about 64.  The rows of one adapter are gathered into
// items of up to `tile` rows, and three kernels share the work:
//  * shrink: a CTA takes an item and one of `splits` parts of K, and writes its
//    share of h, fp32, into the workspace.  x and A pass through a ring of stages of
//    128 k by TMA (A's rows as a box, x's as a box where they lie in a row, else
//    gathered four to a copy) and are multiplied by tcgen05 (M = 128 rows of x, of
//    which the item fills some, N = all ranks of all slices) into tensor memory, so
//    that no warp touches an operand.
//  * join (many rows and more than 64 ranks; else expand does it itself): adds up the shares of
//    h, a warp to a row, and leaves the rows as the fragments that expand multiplies.
//    (Done by every CTA of expand for its rows, it took 10 of 17 us of 1570 rows on
//    q|k|v with rank 64: some 180 instructions for 4 ranks.)
//  * expand: a CTA takes an item and one of `parts` parts of the columns.  It is a
//    programmatic dependent of the one before, and that of shrink, which releases it once
//    it has waited for the kernel before itself: so expand sorts the rows and asks for
//    y and B while they still run, and waits only before it reads h.
// Which rows belong to which adapter is found by every CTA itself, for a scope of up
// to 1024 rows: a histogram of ids in shared memory, a prefix sum over the adapters,
// and the rows of the item in order by a second one (up to 32 rows: matches within a
// warp).  Any mix of ids is served.
//
// expand's products are mma.sync m16n8k16 (490 TFLOP/s measured; the second product
// needs half of that where y streams at 6 TB/s and the rank is 64).  The order of k
// inside a product is free, so lane t of a quad takes 16 contiguous bytes of a row
// and treats them as the k indexes of two products: fragments are single 16-byte
// loads.  B's fragments of 32 columns stay in registers over all rows of the item,
// with ranks up to 32 the next columns' on the way.  The order of columns inside the
// four products is chosen so that a lane holds 8 neighbouring ones of two rows; its 16
// bytes of y come ahead through a ring of its own by cp.async.
//
// Numerics: x and A are binary16, h and the sums fp32 (K in a fixed order).  h is
// multiplied by s_a, scaled by a power of two to the row's largest in
// [2^12, 2^13), and split into two binary16 numbers hi + lo: the second product
// then sees h to 2^-22 of the row's largest instead of 2^-11, for one product
// more.  y + delta is rounded once.
#include "common.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kScope = 1024;        // rows whose ids a CTA sorts
constexpr int kFewRows = 32;        // rows that a warp sorts
constexpr int kFewOfItem = 16;      // rows that shrink multiplies by mma.sync,
constexpr int kFewRanks = 96;       // with up to so many ranks in all, or where no item of a call has more rows (64 rows of
                                    // 32 adapters on q|k|v, us by mma.sync and by tcgen05: 96 ranks 14.4, 14.9; 192 24.1, 18.8)
constexpr int kMaxAdapters = 4096;  // buckets of the histogram
constexpr int kMaxSlices = 4;
constexpr int kMaxRank = 128;
constexpr int kMaxSplits = 8;
constexpr int kColBlock = 32;  // columns of a warp's step
constexpr int kHalfK = 64, kStageK = 2 * kHalfK;  // k of a stage of shrink's ring: two halves of 128-byte rows
constexpr int kMostStages = 8;
constexpr int kBoxRows = 64;  // rows of x in one copy, where they lie in a row (a copy takes some 70 ns to issue, whatever its
                              // size; with 8 rows to a copy 1500 rows of K 11008, rank 128, took 37.6 us for 31.7)
constexpr int kSmemOfTwo = 104 * 1024, kSmemOfOne = 216 * 1024;  // dynamic shared memory of two CTAs on an SM, and of one
constexpr int kSmsOfPlan = 152;  // (the plan does not depend on the device, nor does a workspace's size)

struct LoraArgs {
    const uint16_t *x, *y, *a, *b;
    uint16_t *out;
    const float *scale;
    const int32_t *ids;
    float *h;           // [splits][M][slices * rank]
    int *splits_of;     // of each scope, written by shrink for join
    uint8_t *frags;     // [M] fragments of h, made by join; null: expand makes its own
    float *invs;        // [M]
    long long x_row, y_row, out_row, a_adapter, b_adapter;
    int M, K, N, adapters, rank, slices;
    int col[kMaxSlices + 1];    // first column of each slice, N at the end
    int block[kMaxSlices + 1];  // column blocks before each slice
    int scope;                  // rows of a scope
    int tile, stile;            // rows of an item: 64 or 32; of shrink's items: 128 or 64
    int ctas;                   // of a scope, in the kernel that is launched
    int shrinkers;              // of them in shrink
    int splits, parts;          // most parts of K, and of an item's columns
    int copy;                   // out is not y: rows without an adapter are copied
    int boxes, box_rows;        // boxes of A's rows, of at most 256, and their rows (whole groups of 8)
    int room, pool;             // bytes of shared memory for shrink's ring; for expand's rings
};

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

// 16 bytes global -> shared, asynchronous; zeros where in is false (p is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const uint16_t *p, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `left` (0 .. 3) of this thread's newest groups are on the way.
__device__ __forceinline__ void copies_wait(int left) {
    switch (left) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}
// 64 columns of four rows of a 2-D map whose box is one row high.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int col, int r0, int r1, int r2, int r3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(col), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
        : "memory");
}

// Exclusive prefix sum of v over the block's threads; total gets the sum.
__device__ __forceinline__ int block_scan(int v, int *scratch, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += w;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    __syncthreads();
    return before + s - v;
}

// The items of a scope: up to `tile` rows of one bucket (an adapter, or none).
struct Sorter {
    int *scratch;   // kWarps ints of shared memory
    int *hist;      // [adapters + 1]: rows of each bucket
    int id[kScope / kThreads];  // buckets of this thread's rows, in order; -1 past the scope
    int items, shrunk;          // of all, of p.tile rows and of p.stile
    int first, mine;            // of `tile` rows: before this thread's buckets; in them
    int tile;
    unsigned leaders, same;     // of few rows: the first of each bucket; the lane's equals
    int row0, nrow, per;
    bool few;

    // Parts of K, and of the columns: as many as give each CTA of shrink, or of expand,
    // one (both kernels come to the same splits).
    __device__ __forceinline__ int splits(const LoraArgs &p) const {
        return max(1, min(p.splits, p.shrinkers / max(shrunk, 1)));
    }
    __device__ __forceinline__ int parts(const LoraArgs &p) const {
        return max(1, min(p.parts, p.ctas / max(items, 1)));
    }

    __device__ __forceinline__ static bool counts(const LoraArgs &p, int b) { return b < p.adapters || (b == p.adapters && p.copy); }

    // Called by every thread of the block, at its start, for items of rows_ rows (p.tile or p.stile).
    __device__ __forceinline__ void begin(const LoraArgs &p, int scope, int rows_) {
        const int tid = threadIdx.x, lane = tid & 31;
        tile = rows_;
        row0 = scope * p.scope;
        nrow = min(p.scope, p.M - row0);
        few = nrow <= kFewRows;
        per = (p.adapters + kThreads) / kThreads;
        const auto bucket = [&](int v, int r) {
            if (r >= nrow) return -1;
            if (v >= p.adapters) atomicExch(&g_bad_index, 1);
            return v < 0 || v >= p.adapters ? p.adapters : v;
        };
        if (few) {
            // Every warp knows all rows: an item to each bucket, in the order of their first rows.
            id[0] = bucket(lane < nrow ? __ldg(p.ids + row0 + lane) : -1, lane);
            same = __match_any_sync(~0u, id[0]);
            leaders = __ballot_sync(~0u, id[0] >= 0 && counts(p, id[0]) && (same & ((1u << lane) - 1u)) == 0u);
            items = shrunk = __popc(leaders);
            return;
        }
        constexpr int kMine = kScope / kThreads;
        int raw[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) raw[i] = tid * kMine + i < nrow ? __ldg(p.ids + row0 + tid * kMine + i) : -1;
        for (int i = tid; i <= p.adapters; i += kThreads) hist[i] = 0;  // (while the ids come)
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            id[i] = bucket(raw[i], tid * kMine + i);
            if (id[i] >= 0) atomicAdd(hist + id[i], 1);
        }
        __syncthreads();
        int both = 0, all;  // items of p.tile rows, and of p.stile << 16 (at most 1025 each)
        for (int i = 0; i < per; ++i) {  // this thread's buckets are in a row
            const int b = tid * per + i;
            if (counts(p, b)) both += (hist[b] + p.tile - 1) / p.tile + ((hist[b] + p.stile - 1) / p.stile << 16);
        }
        const int before = block_scan(both, scratch, all), shift = tile == p.stile ? 16 : 0;
        items = all & 0xFFFF;
        shrunk = all >> 16;
        first = before >> shift & 0xFFFF;
        mine = both >> shift & 0xFFFF;
    }

    // The rows and the bucket of an item; called by every thread, ends with a barrier.
    // unit: 3 ints of shared memory.
    __device__ __forceinline__ int item(const LoraArgs &p, int item, int *rows, int *unit, int &n) {
        const int tid = threadIdx.x, lane = tid & 31;
        if (few) {
            unsigned left = leaders;
            for (int i = 0; i < item; ++i) left &= left - 1u;
            const int lead = __ffs(left) - 1;
            const int bucket = __shfl_sync(~0u, id[0], lead);
            const unsigned its = __shfl_sync(~0u, same, lead);
            n = __popc(its);
            if (tid < 32 && its >> lane & 1u) rows[__popc(its & ((1u << lane) - 1u))] = row0 + lane;
            __syncthreads();
            return bucket;
        }
        constexpr int kMine = kScope / kThreads;
        if (item >= first && item < first + mine) {
            int at = first;
            for (int i = 0; i < per; ++i) {
                const int b = tid * per + i;
                if (counts(p, b)) {
                    const int c = (hist[b] + tile - 1) / tile;
                    if (item >= at && item < at + c) {
                        unit[0] = b;
                        unit[1] = (item - at) * tile;
                        unit[2] = min(tile, hist[b] - (item - at) * tile);
                    }
                    at += c;
                }
            }
        }
        __syncthreads();
        const int bucket = unit[0];
        n = unit[2];
        int hits = 0, total;
#pragma unroll
        for (int i = 0; i < kMine; ++i) hits += id[i] == bucket;
        int at = block_scan(hits, scratch, total) - unit[1];
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (id[i] == bucket) {
                if (at >= 0 && at < n) rows[at] = row0 + tid * kMine + i;
                ++at;
            }
        __syncthreads();
        return bucket;
    }
};

// ---- shrink ----

// Shared-memory operand of 128-byte rows, K-major, 128-byte swizzle (8 rows to 1024 bytes).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// D[tmem] (+)= A B^T, M = 128, N = n, K = 16, binary16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, int n, bool add) {
    const uint32_t idesc = 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add));
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 8 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load8(uint32_t addr, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(addr));
}

__host__ __device__ constexpr int tmem_columns(int ranks) {
    return ranks <= 32 ? 32 : ranks <= 64 ? 64 : ranks <= 128 ? 128 : ranks <= 256 ? 256 : 512;
}

// Items of up to 16 rows: the products of tcgen05 cost 150 cycles each whatever the
// rows, so a few rows are multiplied by mma.sync (ranks as M, rows as N), with
// operands loaded straight from global memory in fragment order: lane t of a quad
// takes 16 contiguous bytes of a row as the k indexes of two products.  The warps
// share the CTA's part of K, blocks kb0 .. kb1 - 1 of 32 k, and add their sums through
// shared memory, 16 * MT ranks at a time.  (64 rows of 25 adapters, 11008 k, rank 32:
// 14.1 us, 17 with tcgen05.)
template <int MT, int NT, int AHEAD>
__device__ __forceinline__ void shrink_few(const LoraArgs &p, const uint16_t *a, const int *rows, int n, int split,
                                           int kb0, int kb1, float *red) {
    constexpr int G = 16 * MT;
    const int F = p.slices * p.rank;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int k0 = kb0 + (kb1 - kb0) * warp / kWarps, k1 = kb0 + (kb1 - kb0) * (warp + 1) / kWarps;
    const uint16_t *xr[NT];
    bool xv[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        xv[i] = 8 * i + g < n;
        xr[i] = p.x + rows[xv[i] ? 8 * i + g : 0] * p.x_row + 8 * t;
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int f0 = 0; f0 < F; f0 += G) {
        float acc[MT][NT][4] = {};
        const uint16_t *ar = a + (long long)(f0 + g) * p.K + 8 * t;
        for (int b = k0; b < k1; b += AHEAD) {
            uint4 av[AHEAD][2 * MT], xf[AHEAD][NT];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const bool in = b + q < k1 && 32 * (b + q) + 8 * t < p.K;
#pragma unroll
                for (int i = 0; i < NT; ++i) xf[q][i] = in && xv[i] ? load16(xr[i] + 32 * (b + q)) : zero;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i)
                    av[q][i] = in && f0 + 8 * i + g < F ? load16(ar + (long long)(8 * i) * p.K + 32 * (b + q)) : zero;
            }
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 u = av[q][2 * m], l = av[q][2 * m + 1];
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_16816(acc[m][i], u.x, l.x, u.y, l.y, xf[q][i].x, xf[q][i].y);
#pragma unroll
                    for (int i = 0; i < NT; ++i) mma_16816(acc[m][i], u.z, l.z, u.w, l.w, xf[q][i].z, xf[q][i].w);
                }
        }
        // red [warp][8 * NT rows][G]
        float *mine = red + warp * 8 * NT * G;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[(8 * i + 2 * t + (e & 1)) * G + 16 * m + g + 8 * (e >> 1)] = acc[m][i][e];
        __syncthreads();
        for (int e = threadIdx.x; e < n * G; e += kThreads) {
            const int r = e / G, f = f0 + e % G;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[w * 8 * NT * G + e];
            if (f < F) p.h[((long long)split * p.M + rows[r]) * F + f] = v;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads, 2) shrink_kernel(const __grid_constant__ CUtensorMap amap,
                                                          const __grid_constant__ CUtensorMap xmap,
                                                          const __grid_constant__ CUtensorMap xbox,
                                                          const __grid_constant__ LoraArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-(uint32_t)__cvta_generic_to_shared(smem_raw) & 1023u);
    __shared__ int scratch[kWarps], rows[128], unit[3];
    __shared__ __align__(8) uint64_t bars[2 * kMostStages + 1];
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    volatile int *abort = &abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = (uint32_t)__cvta_generic_to_shared(bars), empty = full + 8 * kMostStages,
                   done = full + 16 * kMostStages;
    const int F = p.slices * p.rank, F16 = (F + 15) / 16 * 16, columns = tmem_columns(F16);
    const bool tensor = p.M > kFewOfItem;  // some item may be of many rows
    if (tid == 0 && tensor) {
        for (int i = 0; i < 2 * kMostStages + 1; ++i) mbar_init(full + 8 * i, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&amap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&xbox) : "memory");
    }
    // (Kept through the wait: the kernel before has its tensor memory already, or, being
    // one that takes it after it released this one, more shared memory than is left beside.)
    if (warp == 2 && tensor) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(&tmem_at)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    pdl_launch_dependents();  // (expand may start: what it reads before its own wait is complete)
    Sorter sorter;
    sorter.scratch = scratch;
    sorter.hist = reinterpret_cast<int *>(smem + p.room);
    sorter.begin(p, blockIdx.x / p.ctas, p.stile);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_at;
    const int kb = (p.K + kStageK - 1) / kStageK, splits = sorter.splits(p);
    if (p.frags && tid == 0 && blockIdx.x % p.ctas == 0) p.splits_of[blockIdx.x / p.ctas] = splits;
    uint32_t stage_no = 0, units = 0;  // stages and items so far: the barriers' phases
    for (int u = blockIdx.x % p.ctas; u < sorter.shrunk * splits; u += p.ctas) {
        int n;
        const int split = u % splits, bucket = sorter.item(p, u / splits, rows, unit, n);
        const int c0 = (int)((long long)kb * split / splits), chunks = (int)((long long)kb * (split + 1) / splits) - c0;
        if (bucket == p.adapters) continue;  // (alike for all threads; rows is written again after a barrier)
        if (n <= kFewOfItem && (F <= kFewRanks || !tensor)) {
            const uint16_t *a = p.a + bucket * p.a_adapter;
            const int b0 = c0 * (kStageK / 32), b1 = min((p.K + 31) / 32, (c0 + chunks) * (kStageK / 32));
            float *red = reinterpret_cast<float *>(smem);
            if (F <= 16) shrink_few<1, 2, 4>(p, a, rows, n, split, b0, b1, red);
            else if (F <= 32) shrink_few<2, 2, 2>(p, a, rows, n, split, b0, b1, red);
            else if (n <= 8) shrink_few<4, 1, 2>(p, a, rows, n, split, b0, b1, red);
            else shrink_few<4, 2, 1>(p, a, rows, n, split, b0, b1, red);
            fence_proxy_async_smem();  // (the next item's copies may come here)
            __syncthreads();
            continue;
        }
        // A stage: A's rows, then x's; the products read 128 rows of x, what lies behind the
        // item's goes into rows of the sums that nobody reads.
        const bool box = n > 16 && rows[n - 1] - rows[0] == n - 1;
        const int xrow = F16, xrows = box ? (n + kBoxRows - 1) / kBoxRows * kBoxRows : (n + 7) / 8 * 8;
        const int half = (xrow + xrows) * 128, stage = 2 * half;
        const int stages = min(kMostStages, (p.room - 128 * 128) / stage);
        const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
        const uint32_t bytes = 2 * (p.boxes * p.box_rows * 128 + (box ? xrows : (n + 3) / 4 * 4) * 128);
        if (warp == 0) {
            for (int c = 0; c < chunks; ++c) {
                const uint32_t i = stage_no + c, b = i % kMostStages, at = base + c % stages * stage;
                // (A slot is free when the stage that last lay in it was read, `stages` ago.)
                if (c >= stages) {
                    const uint32_t last = i - stages;
                    mbar_wait(empty + 8 * (last % kMostStages), last / kMostStages & 1, abort);
                }
                const int k = (c0 + c) * kStageK;
                if (lane == 0) mbar_expect_tx(full + 8 * b, bytes);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kh = k + kHalfK * h;
                    const uint32_t to = at + h * half, bar = full + 8 * b;
                    if (lane >= 32 - p.boxes) {
                        const int row = (lane - (32 - p.boxes)) * p.box_rows;  // (rows past F are zero, and end before x's)
                        tma_load_3d(to + row * 128, &amap, kh, row, bucket, bar);
                    }
                    if (box) {  // (what lies behind the item's rows is read too, and zero behind the last of all)
                        if (kBoxRows * lane < n)
                            tma_load_2d(to + (xrow + kBoxRows * lane) * 128, &xbox, kh, rows[0] + kBoxRows * lane, bar);
                    } else if (4 * lane < n) {
                        const int end = n - 1;
                        tma_gather4(to + (xrow + 4 * lane) * 128, &xmap, kh, rows[4 * lane], rows[min(4 * lane + 1, end)],
                                    rows[min(4 * lane + 2, end)], rows[min(4 * lane + 3, end)], bar);
                    }
                }
            }
        } else if (warp == 1 && lane == 0) {
            for (int c = 0; c < chunks; ++c) {
                const uint32_t i = stage_no + c, b = i % kMostStages, at = base + c % stages * stage;
                if (!mbar_wait(full + 8 * b, i / kMostStages & 1, abort)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int k = 0; k < kStageK / 16; ++k) {
                    const uint32_t from = at + k / 4 * half + k % 4 * 32;
                    const uint64_t x = operand_desc(from + xrow * 128), a = operand_desc(from);
                    mma_f16(tmem, x, a, min(F16, 256), c > 0 || k > 0);
                    if (F16 > 256) mma_f16(tmem + 256, x, operand_desc(from + 256 * 128), F16 - 256, c > 0 || k > 0);
                }
                mma_commit(empty + 8 * b);
            }
            mma_commit(done);
        }
        __syncwarp();
        // Every stage is read before the next item's copies come (the products are in order).
        const bool ok = mbar_wait(done, units & 1, abort);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // The sums go out row by row through the ring's place (rows 16 bytes longer than their data).
        const int r = 32 * warp + lane, pitch = 4 * F + 16;
        if (32 * warp < n) {
            for (int f = 0; f < F; f += 32) {
                float v[4][8];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (f + 8 * q < F) tmem_load8(tmem + ((uint32_t)(32 * warp) << 16) + f + 8 * q, v[q]);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int q = 0; q < 4; ++q) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) asm volatile("" : "+f"(v[q][i]));  // (used after the wait)
                    if (f + 8 * q < F) {
                        float4 *to = reinterpret_cast<float4 *>(smem + r * pitch + 4 * (f + 8 * q));
                        to[0] = make_float4(v[q][0], v[q][1], v[q][2], v[q][3]);
                        to[1] = make_float4(v[q][4], v[q][5], v[q][6], v[q][7]);
                    }
                }
            }
            fence_proxy_async_smem();
            if (r < n && ok) {
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                                 p.h + ((long long)split * p.M + rows[r]) * F),
                             "r"(base + r * pitch), "r"(4 * F)
                             : "memory");
                bulk_commit_group();
                bulk_wait_group<0>();
            }
        }
        stage_no += chunks;  // (at least one)
        ++units;
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    __syncthreads();
    if (warp == 2 && tensor) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

// ---- expand ----

// mma_16816 from sums of zero.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The fragments of the second product: for each row, block of 16 ranks and lane t
// of a quad, the 16 bytes {hi, hi, lo, lo} of 4 ranks in a row, two to a word.  Rows
// are `pitch` bytes apart, an odd number of 64, so that 8 lanes of a load meet no
// bank twice.
template <int RK>
__host__ __device__ constexpr int frag_pitch(int slices) {
    return slices * RK * 4 % 128 == 0 ? slices * RK * 4 + 64 : slices * RK * 4;
}
// Byte offset in a row of ranks r .. r + 3 (r a multiple of 4) of slice s.
template <int RK>
__device__ __forceinline__ int frag_at(int s, int r) {
    // Of 16 ranks lane t holds 4t .. 4t + 3; of 32, 8t .. 8t + 7, for two products.
    const int k16 = RK == 16 ? 0 : 2 * (r >> 5) + (r >> 2 & 1), t = RK == 16 ? r >> 2 : r >> 3 & 3;
    return ((s * (RK / 16) + k16) * 4 + t) * 16;
}

// Sum of the shares of 4 ranks.
__device__ __forceinline__ float4 add_shares(const float *src, long long share, int splits) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < splits; c += 4) {
        float4 part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // (written by the kernel before: no read-only loads)
            part[i] = c + i < splits ? __ldcg(reinterpret_cast<const float4 *>(src + (c + i) * share))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.x += part[i].x;
            v.y += part[i].y;
            v.z += part[i].z;
            v.w += part[i].w;
        }
    }
    return v;
}
// Bits of the largest finite one of four values, which order as they do.  (What is not
// finite stays so under any power of two, and sets none: a row's other ranks and slices are
// scaled as without it.)
__device__ __forceinline__ int top_of(const float4 &v) {
    const auto bits = [](float x) {
        const int b = __float_as_int(fabsf(x));
        return b < 0x7F800000 ? b : 0;
    };
    return max(max(bits(v.x), bits(v.y)), max(bits(v.z), bits(v.w)));
}
// Power of two of a row: 12 - x for a largest value (its bits) in [2^x, 2^(x + 1)); 0 for
// rows of zeros.
__device__ __forceinline__ int shift_of(int top) {
    const int x = (top >> 23) - 127;
    return top == 0 ? 0 : 12 - max(x, -100);
}
__device__ __forceinline__ uint4 fragment(const float4 &v, float up) {
    const float a = v.x * up, b = v.y * up, c = v.z * up, d = v.w * up;
    const uint32_t h0 = pack(a, b), h1 = pack(c, d);
    const float2 f0 = unpack(h0), f1 = unpack(h1);
    const auto rest = [](float x, float hi) { return fabsf(x - hi) < 1e30f ? x - hi : 0.f; };  // (none of infinities)
    return make_uint4(h0, h1, pack(rest(a, f0.x), rest(b, f0.y)), pack(rest(c, f1.x), rest(d, f1.y)));
}

// A warp to a row: the fragments of h, rows of slices * RK * 4 bytes.
template <int RK>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ LoraArgs p) {
    pdl_launch_dependents();  // (what expand reads before its wait was complete before shrink released this kernel)
    const int R = p.slices * RK, F = p.slices * p.rank, lane = threadIdx.x & 31;
    const int m = blockIdx.x * kWarps + (int)(threadIdx.x >> 5);
    const int id = m < p.M ? __ldg(p.ids + m) : -1;
    const bool none = id < 0 || id >= p.adapters;
    const float scale = none || !p.scale ? 1.f : __ldg(p.scale + id);
    pdl_wait();
    if (none) return;
    const int splits = __ldcg(p.splits_of + m / p.scope);
    constexpr int J = (kMaxSlices * RK + 127) / 128;  // groups of 4 ranks of a lane
    float4 v[J];
    int top = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int r = 128 * j + 4 * lane;
        v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < R && r % RK < p.rank) {  // (ranks past the adapters' are zero)
            v[j] = add_shares(p.h + (long long)m * F + r / RK * p.rank + r % RK, (long long)p.M * F, splits);
            v[j] = make_float4(v[j].x * scale, v[j].y * scale, v[j].z * scale, v[j].w * scale);
        }
        top = max(top, top_of(v[j]));
    }
    top = __reduce_max_sync(~0u, top);
    const int shift = shift_of(top);
    if (lane == 0) p.invs[m] = __int_as_float((127 - shift) << 23);
    uint8_t *dst = p.frags + (long long)m * R * 4;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int r = 128 * j + 4 * lane;
        if (r < R) *reinterpret_cast<uint4 *>(dst + frag_at<RK>(r / RK, r % RK)) = fragment(v[j], __int_as_float((127 + shift) << 23));
    }
}

// The fragments of the item's rows that join made.  Ends with a barrier.
template <int RK>
__device__ __forceinline__ void load_fragments(const LoraArgs &p, const int *rows, int n, uint8_t *smem, float *inv) {
    const int G = p.slices * RK / 4, pitch = frag_pitch<RK>(p.slices);
    const uint32_t by = ((1u << 22) + G - 1) / G, base = (uint32_t)__cvta_generic_to_shared(smem);
    for (int e = threadIdx.x; e < n * G; e += kThreads) {
        const int row = (int)(e * by >> 22), at = 16 * (e - row * G);
        copy16(base + row * pitch + at, reinterpret_cast<const uint16_t *>(p.frags + (long long)rows[row] * G * 16 + at), true);
    }
    copies_commit();
    if (threadIdx.x < n) inv[threadIdx.x] = __ldcg(p.invs + rows[threadIdx.x]);
    copies_wait(0);
    __syncthreads();
}

// Adds up the shares of h of the item's rows, scales and splits them into fragments.
// The sums, 4 ranks of a row to a thread, first lie where their fragments will; tops
// holds the bits of each row's largest finite value, which order as the values do,
// and is zero on entry.  Ends with a barrier.
template <int RK>
__device__ __forceinline__ void gather_h(const LoraArgs &p, float scale, int splits, const int *rows, int n,
                                         uint8_t *smem, int *tops, float *inv) {
    const int G = p.slices * RK / 4, F = p.slices * p.rank, pitch = frag_pitch<RK>(p.slices);
    const uint32_t by = ((1u << 22) + G - 1) / G;  // e / G = e * by >> 22 for e < 2^13
    const long long share = (long long)p.M * F;
    constexpr int W = RK / 4;  // W lanes in a row hold a row's ranks of a slice
    for (int e0 = threadIdx.x; e0 < (n * G + 31) / 32 * 32; e0 += kThreads) {
        const int row = (int)(e0 * by >> 22), r = 4 * (e0 - row * G);
        const bool in = e0 < n * G;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (in && r % RK < p.rank) {  // (ranks past the adapters' are zero)
            v = add_shares(p.h + (long long)rows[row] * F + r / RK * p.rank + r % RK, share, splits);
            v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
        }
        int top = top_of(v);
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        if (in) {
            *reinterpret_cast<float4 *>(smem + row * pitch + frag_at<RK>(r / RK, r % RK)) = v;
            if (r % RK == 0) atomicMax(tops + row, top);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n * G; e += kThreads) {
        const int row = (int)(e * by >> 22), r = 4 * (e - row * G), shift = shift_of(tops[row]);
        if (r == 0) inv[row] = __int_as_float((127 - shift) << 23);
        uint4 *at = reinterpret_cast<uint4 *>(smem + row * pitch + frag_at<RK>(r / RK, r % RK));
        *at = fragment(*reinterpret_cast<const float4 *>(at), __int_as_float((127 + shift) << 23));
    }
    __syncthreads();
}

// Where a warp stands among the column blocks.
struct Columns {
    int blk, next;  // block; first one of the next slice
    int col, end;   // first column of the block; end of its slice
    int slice;
    __device__ __forceinline__ void start(const LoraArgs &p, int b) {
        blk = b;
        slice = 0;
        while (slice + 1 < p.slices && blk >= p.block[slice + 1]) ++slice;
        next = p.block[slice + 1];
        col = p.col[slice] + (blk - p.block[slice]) * kColBlock;
        end = p.col[slice + 1];
    }
    __device__ __forceinline__ void step(const LoraArgs &p) {
        blk += kWarps;
        col += kWarps * kColBlock;
        if (blk >= next) start(p, blk);
    }
};

// out = y + h B^T over the CTA's column blocks [b0, b1) of the item's rows, whose
// addresses in y and out are yrow and orow.  ready() is called by every thread once
// the first copies are on their way; it leaves the fragments and inv in place.
template <int RK, class Ready>
__device__ __forceinline__ void expand(const LoraArgs &p, const uint16_t *bw, const uint16_t *const *yrow,
                                       uint16_t *const *orow, int n, uint8_t *smem, const float *inv, int b0, int b1,
                                       Ready ready) {
    constexpr int KS = RK / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tiles = (n + 15) / 16, pitch = frag_pitch<RK>(p.slices);
    const uint32_t frag = (uint32_t)__cvta_generic_to_shared(smem) + g * pitch + 16 * t;
    // The warp's ring of y: `depth` column blocks of up to 64 rows, 16 bytes a lane each.
    const int slot = tiles * 1024, depth = min(4, p.pool / (kWarps * slot));
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + p.tile * pitch) + warp * depth * slot + lane * 16;
    const uint32_t ring_end = ring + depth * slot;
    Columns ahead, own;
    own.start(p, b0 + warp);
    ahead = own;
    auto copy_y = [&](uint32_t dst) {
        if (ahead.blk < b1 && ahead.col + 8 * t < ahead.end) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (g + 8 * q < n) copy16(dst + q * 512, yrow[g + 8 * q] + ahead.col + 8 * t, true);
        }
        copies_commit();
        ahead.step(p);
    };
    // Column (product j, n = g) is col + 8 (g / 2) + 2 j + g % 2.
    uint32_t bf[4][KS][2];
    auto load_b = [&](const Columns &at) {
        const int c0 = at.col + 8 * (g >> 1) + (g & 1);
        const uint16_t *row = bw + (long long)c0 * p.rank;
#pragma unroll
        for (int j = 0; j < 4; ++j, row += 2 * p.rank) {
            const bool in = c0 + 2 * j < at.end;
            if (RK == 16) {
                uint2 v = make_uint2(0u, 0u);
                if (in && 4 * t < p.rank) v = __ldg(reinterpret_cast<const uint2 *>(row + 4 * t));
                bf[j][0][0] = v.x;
                bf[j][0][1] = v.y;
            } else {
#pragma unroll
                for (int q = 0; q < KS / 2; ++q) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (in && 32 * q + 8 * t < p.rank) v = load16(row + 32 * q + 8 * t);
                    bf[j][2 * q][0] = v.x;
                    bf[j][2 * q][1] = v.y;
                    bf[j][2 * q + 1][0] = v.z;
                    bf[j][2 * q + 1][1] = v.w;
                }
            }
        }
    };
    if (own.blk < b1) load_b(own);
    for (int d = 0; d < depth; ++d) copy_y(ring + d * slot);
    ready();
    if (own.blk >= b1) {
        copies_wait(0);
        return;
    }
    uint32_t at = ring;
    while (true) {
        copies_wait(depth - 1);  // (a lane reads only what it copied itself)
        const uint32_t f0 = frag + own.slice * (64 * KS);
        const int col = own.col + 8 * t;
        const bool cv = col < own.end;
        for (int tile = 0; tile < tiles; ++tile) {
            const uint4 old[2] = {lds128(at + 2 * tile * 512), lds128(at + (2 * tile + 1) * 512)};
            const uint32_t row = f0 + 16 * tile * pitch;
            float acc[4][4];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint4 u = lds128(row + 64 * k), l = lds128(row + 8 * pitch + 64 * k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (k == 0) mma_first(acc[j], u.x, l.x, u.y, l.y, bf[j][k][0], bf[j][k][1]);
                    else mma_16816(acc[j], u.x, l.x, u.y, l.y, bf[j][k][0], bf[j][k][1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_16816(acc[j], u.z, l.z, u.w, l.w, bf[j][k][0], bf[j][k][1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * tile + 8 * i + g;
                const float f = inv[r];
                const uint32_t v[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 y = unpack(v[j]);
                    o[j] = pack(fmaf(acc[j][2 * i], f, y.x), fmaf(acc[j][2 * i + 1], f, y.y));
                }
                uint16_t *dst = orow[r] + col;
                if (cv && r < n) *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
        own.step(p);
        if (own.blk >= b1) break;
        load_b(own);
        copy_y(at);
        at = at + slot == ring_end ? ring : at + slot;
    }
    copies_wait(0);
}

// Rows without an adapter, where out is not y: the CTA's columns are copied.
__device__ __forceinline__ void copy_rows(const LoraArgs &p, const int *rows, int n, int c0, int c1) {
    const int units = (c1 - c0) / 8;
    for (int e = threadIdx.x; e < units * n; e += kThreads) {
        const int r = rows[e / units], c = c0 + e % units * 8;
        *reinterpret_cast<uint4 *>(p.out + r * p.out_row + c) = *reinterpret_cast<const uint4 *>(p.y + r * p.y_row + c);
    }
}

template <int RK>
__global__ void __launch_bounds__(kThreads, 2) expand_kernel(const __grid_constant__ LoraArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scratch[kWarps], rows[64], unit[3];
    __shared__ float inv[64];
    __shared__ int tops[64];
    __shared__ const uint16_t *yrow[64];
    __shared__ uint16_t *orow[64];
    const int tid = threadIdx.x;
    Sorter sorter;
    sorter.scratch = scratch;
    sorter.hist = reinterpret_cast<int *>(smem + p.tile * frag_pitch<RK>(p.slices) + p.pool);
    // (What is read before the wait was complete before shrink released its dependent.)
    sorter.begin(p, blockIdx.x / p.ctas, p.tile);
    const int splits = sorter.splits(p), parts = sorter.parts(p);
    bool waited = false;
    for (int u = blockIdx.x % p.ctas; u < sorter.items * parts; u += p.ctas) {
        int n;
        const int part = u % parts, bucket = sorter.item(p, u / parts, rows, unit, n);
        if (bucket == p.adapters) {
            if (!waited) pdl_wait();
            waited = true;
            const int units = p.N / 8;
            copy_rows(p, rows, n, 8 * (int)((long long)units * part / parts),
                      8 * (int)((long long)units * (part + 1) / parts));
        } else {
            const int blocks = p.block[p.slices];
            const int b0 = (int)((long long)blocks * part / parts), b1 = (int)((long long)blocks * (part + 1) / parts);
            const uint16_t *bw = p.b + bucket * p.b_adapter;
            if (tid == 0 && b0 < b1) {  // B's rows of these columns, on their way into L2
                Columns first, last;
                first.start(p, b0);
                last.start(p, b1 - 1);
                const int end = min(last.col + kColBlock, last.end);
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(bw + (long long)first.col * p.rank),
                             "r"((end - first.col) * p.rank * 2));
            }
            if (tid < 64) tops[tid] = 0;
            if (tid < n) {
                yrow[tid] = p.y + rows[tid] * p.y_row;
                orow[tid] = p.out + rows[tid] * p.out_row;
            }
            __syncthreads();
            expand<RK>(p, bw, yrow, orow, n, smem, inv, b0, b1, [&] {
                if (!waited) pdl_wait();
                waited = true;
                if (p.frags) load_fragments<RK>(p, rows, n, smem, inv);
                else gather_h<RK>(p, p.scale ? __ldg(p.scale + bucket) : 1.f, splits, rows, n, smem, tops, inv);
            });
        }
        __syncthreads();
    }
    if (!waited) pdl_wait();  // (the kernel after this one counts on the others' end)
}

int round_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// How a call is cut: from its arguments alone, for the workspace's size.
struct Cut {
    int scopes, scope, tile, stile, shrinkers, expanders, splits, parts, room;
};
Cut cut_of(const f16_adapters *s, int M, int blocks) {
    Cut c;
    c.scopes = (int)((M + (long long)kScope - 1) / kScope);
    c.scope = (M + c.scopes - 1) / c.scopes;
    c.tile = round_rank(s->rank) * s->slices <= 384 ? 64 : 32;
    // Parts of K of a stage or more, parts of the columns of a block for each warp.
    const int kb = (s->K + kStageK - 1) / kStageK;
    c.splits = kb < kMaxSplits ? kb : kMaxSplits;
    // shrink's ring: as many stages as fit an item's rows, up to 8, and room behind the last one
    // for the 128 rows of x that a product reads.  Two CTAs on an SM where two stages of the
    // largest item fit that, and the sums, else one.  (shrink_few needs 32 KB of it.)
    const int F = s->rank * s->slices, hist = (s->adapters + 1) * 4;
    c.stile = F <= 192 ? 128 : 64;
    const int stage = 2 * ((F + 15) / 16 * 16 + c.stile) * 128, tail = 128 * 128;
    const bool two = (2 * stage + tail > 4 * c.stile * (F + 4) ? 2 * stage + tail : 4 * c.stile * (F + 4)) + hist <= kSmemOfTwo && tmem_columns((F + 15) / 16 * 16) <= 256;
    c.room = (two ? kSmemOfTwo : kSmemOfOne) - hist;
    c.parts = (blocks + kWarps - 1) / kWarps;
    // As many CTAs as the SMs hold, shared by the scopes, but one for each item where the rows lie
    // in runs, and no more than there can be work for.
    const long long full = (c.scope + c.tile - 1) / c.tile;
    const long long items = c.scope < full + s->adapters + 1 ? c.scope : full + s->adapters + 1;
    const auto ctas = [&](long long on_sm, long long rows, long long parts) {
        const long long share = on_sm * kSmsOfPlan / c.scopes, least = (c.scope + rows - 1) / rows + 3,
                        most = items * parts;
        const long long n = share > least ? share : least;
        return (int)(n < most ? n : most);
    };
    c.shrinkers = ctas(two ? 2 : 1, c.stile, c.splits);
    c.expanders = ctas(2, c.tile, c.parts);
    return c;
}

}  // namespace

// Reads and clears this translation unit's records: bit 0 an expired wait, bit 1 a bad index.
int lora_status() {
    int w = 0, b = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&w, g_wait_expired, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&b, g_bad_index, sizeof(int)) != cudaSuccess)
        return -1;
    if (w) cudaMemcpyToSymbol(g_wait_expired, &zero, sizeof(int));
    if (b) cudaMemcpyToSymbol(g_bad_index, &zero, sizeof(int));
    return (w ? 1 : 0) | (b ? 2 : 0);
}
}  // namespace w4a16

using namespace w4a16;

namespace {

// Host checks of the adapters; fills the columns' part of p.
int check_adapters(const f16_adapters *s, LoraArgs &p) {
    if (!s) return W4_ERR_NULL;
    if (s->adapters < 1 || s->adapters > kMaxAdapters || s->rank < 8 || s->rank > kMaxRank || s->rank % 8 != 0 ||
        s->K < 8 || s->K % 8 != 0 || s->N < 8 || s->N % 8 != 0 || s->slices < 1 || s->slices > kMaxSlices)
        return W4_ERR_SHAPE;
    for (int i = 0; i < s->slices; ++i) {
        p.col[i + 1] = s->columns[i];
        if (s->columns[i] <= p.col[i] || s->columns[i] % 8 != 0) return W4_ERR_SHAPE;
        p.block[i + 1] = p.block[i] + (p.col[i + 1] - p.col[i] + kColBlock - 1) / kColBlock;
    }
    return p.col[s->slices] == s->N ? W4A16_OK : W4_ERR_SHAPE;
}

// A launch as a programmatic dependent.
template <class K, class... A>
int launch(K kernel, long long ctas, int smem, void *stream, const A &...args) {
    if (ctas > 0x7FFFFFFFll) return W4_ERR_SHAPE;
    if (!ensure_smem(reinterpret_cast<const void *>(kernel), smem)) return W4_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return W4_ERR_LAUNCH;
    }
    return W4A16_OK;
}

}  // namespace

namespace {

// Whether join runs: where there are more ranks than 64 for many rows.  (1570 rows on
// q|k|v, rank 64: 23.5 us with it, 33.5 without; on gate|up, rank 16: 47.4 and 43.0.)
bool joined(const f16_adapters *s, int M) { return M > kFewRows && s->slices * s->rank > 64; }

// The workspace: the shares of h, then what join leaves.
struct Workspace {
    size_t frags, invs, splits_of, bytes;
};
Workspace workspace_of(const f16_adapters *s, int M, const Cut &c) {
    Workspace w;
    const size_t rows = (size_t)M;
    w.frags = c.splits * rows * s->slices * s->rank * 4;  // (multiples of 32 bytes)
    w.invs = w.frags + (joined(s, M) ? rows * s->slices * round_rank(s->rank) * 4 : 0);
    w.splits_of = w.invs + (joined(s, M) ? rows * 4 : 0);
    w.bytes = w.splits_of + (joined(s, M) ? (size_t)c.scopes * 4 : 0);
    return w;
}

}  // namespace

extern "C" size_t f16_lora_workspace_bytes(const f16_adapters *s, int M) {
    LoraArgs p = {};
    if (M < 1 || check_adapters(s, p) != W4A16_OK) return 0;
    return workspace_of(s, M, cut_of(s, M, p.block[s->slices])).bytes;
}

extern "C" int f16_lora(const uint16_t *x, int64_t x_row, const uint16_t *y, int64_t y_row, uint16_t *out,
                        int64_t out_row, const f16_adapters *s, const int32_t *ids, int M, void *workspace,
                        size_t workspace_bytes, void *stream) {
    LoraArgs p = {};
    int st = check_adapters(s, p);
    if (st != W4A16_OK) return st;
    if (M < 0) return W4_ERR_SHAPE;
    if (M == 0) return W4A16_OK;
    if (!x || !y || !out || !ids || !s->a || !s->b) return W4_ERR_NULL;
    const auto stride_ok = [](int64_t v) { return v > 0 && v % 8 == 0; };
    if (!aligned16(x) || !aligned16(y) || !aligned16(out) || !aligned16(s->a) || !aligned16(s->b) ||
        (reinterpret_cast<uintptr_t>(ids) & 3u) != 0 || (reinterpret_cast<uintptr_t>(s->scale) & 3u) != 0 ||
        !stride_ok(x_row) || !stride_ok(y_row) || !stride_ok(out_row) || !stride_ok(s->a_adapter) ||
        !stride_ok(s->b_adapter))
        return W4_ERR_ALIGN;
    if (M > 1 && out_row < s->N) return W4_ERR_SHAPE;
    const Cut c = cut_of(s, M, p.block[s->slices]);
    const Workspace ws = workspace_of(s, M, c);
    if (!workspace || workspace_bytes < ws.bytes) return W4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4_ERR_ALIGN;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    p.x = x;
    p.y = y;
    p.a = s->a;
    p.x_row = x_row;
    p.a_adapter = s->a_adapter;
    p.out = out;
    p.b = s->b;
    p.scale = s->scale;
    p.ids = ids;
    uint8_t *const work = static_cast<uint8_t *>(workspace);
    p.h = reinterpret_cast<float *>(work);
    p.frags = joined(s, M) ? work + ws.frags : nullptr;
    p.invs = reinterpret_cast<float *>(work + ws.invs);
    p.splits_of = reinterpret_cast<int *>(work + ws.splits_of);
    p.y_row = y_row;
    p.out_row = out_row;
    p.b_adapter = s->b_adapter;
    p.M = M;
    p.K = s->K;
    p.N = s->N;
    p.adapters = s->adapters;
    p.rank = s->rank;
    p.slices = s->slices;
    p.scope = c.scope;
    p.tile = c.tile;
    p.stile = c.stile;
    p.shrinkers = p.ctas = c.shrinkers;
    p.splits = c.splits;
    p.parts = c.parts;
    p.copy = out != y || out_row != y_row;
    const int rk = round_rank(s->rank), F = s->rank * s->slices, hist = (s->adapters + 1) * 4;
    // A as [adapters][slices * rank][K], boxes of 64 k and all rows (two boxes of more
    // than 256); x as [M][K], boxes of 64 k of one row, copied four at a time, and of kBoxRows.
    // (None is used where every item has few rows.)
    CUtensorMap amap = {}, xmap = {}, xbox = {};
    p.boxes = F > 256 ? 2 : 1;
    p.box_rows = p.boxes == 1 ? F : (F / 2 + 7) / 8 * 8;
    const uint64_t x_bytes = 2ull * (M > 1 ? x_row : s->K);
    if (M > kFewOfItem &&
        (!make_map_3d(&amap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, s->a, (uint64_t)s->K, (uint64_t)F, (uint64_t)s->adapters,
                     2ull * s->K, 2ull * (s->adapters > 1 ? s->a_adapter : 8), kHalfK, (uint32_t)p.box_rows, 1,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)s->K, (uint64_t)M, x_bytes, kHalfK, 1,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_map_2d(&xbox, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)s->K, (uint64_t)M, x_bytes, kHalfK, kBoxRows,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
        return encode_fn() ? W4_ERR_SHAPE : W4_ERR_DEVICE;
    p.room = c.room;
    st = launch(shrink_kernel, (long long)c.scopes * c.shrinkers, p.room + hist + 1024, stream, amap, xmap, xbox, p);
    if (st != W4A16_OK) return st;
    if (p.frags) {
        const auto join = rk == 16 ? join_kernel<16> : rk == 32 ? join_kernel<32> : rk == 64 ? join_kernel<64> : join_kernel<128>;
        st = launch(join, ((long long)M + kWarps - 1) / kWarps, 0, stream, p);
        if (st != W4A16_OK) return st;
    }
    // expand: the fragments, and rings of up to three column blocks for each warp.
    const int frag = c.tile * (rk == 16   ? frag_pitch<16>(s->slices)
                               : rk == 32 ? frag_pitch<32>(s->slices)
                               : rk == 64 ? frag_pitch<64>(s->slices)
                                          : frag_pitch<128>(s->slices));
    const int block = kWarps * c.tile * 64;  // one block a warp
    int depth = 3;
    while (depth > 1 && frag + depth * block + hist > kSmemOfTwo) --depth;
    p.pool = depth * block;
    p.ctas = c.expanders;
    const auto kernel = rk == 16 ? expand_kernel<16> : rk == 32 ? expand_kernel<32> : rk == 64 ? expand_kernel<64>
                                                                                              : expand_kernel<128>;
    return launch(kernel, (long long)c.scopes * c.expanders, frag + p.pool + hist, stream, p);
}
