// How f16_attention shares its work out, common to its kernels.
//
// The query rows of one sequence and key/value head are its new tokens times
// the head's query heads: row r is token r / G of the sequence, query head
// r % G of the group (G = q_heads / kv_heads).  An item is a tile of `rows`
// such rows (of one sequence, one key/value head) with the range of
// positions [lo, hi) that any of its rows sees; a unit is one tile of `keys`
// positions of that range.  All items' units, in the order (sequence, head,
// row tile, key tile), are cut into one contiguous range per CTA, equal to
// within a unit, whatever the lengths.  An item cut by a range boundary is
// computed in parts: each part's CTA leaves its unnormalised output, running
// maximum and sum in the workspace, and a second kernel joins them.  Every
// CTA works its range out from the lengths by itself: the host needs no
// lengths, and the split depends on nothing but the batch, so results repeat.
#pragma once

#include "kv.cuh"

namespace w4a16 {

struct AttnArgs {
    KvBatch b;
    const uint16_t *q;
    uint16_t *y;
    float *lse;
    long long q_token, q_head, y_token, y_head;
    int group, kv_heads, head_dim;
    int causal, window;
    int num_pages, page_size, box_rows;
    int few_tiles;  // a sequence is expected to have few row tiles (chooses how the plan is summed)
    float scale;    // times log2(e): the softmax is taken in powers of two
    float *part_o;  // [2 * grid][rows][head_dim]
    float *part_ml; // [2 * grid][rows][2]: running maximum (base-2 scaled scores) and sum
    struct JoinItem *joins;  // [grid]
};

// An item that starts in the range of CTA c and is finished by later CTAs:
// parts at slots 2c + 1, 2(c + 1), 2(c + 2), ...
struct JoinItem {
    int parts;  // 0: none
    int q0;     // first token of the sequence
    int head;   // key/value head
    int row0, rows;
};

struct Item {
    int nrt;     // row tiles of the sequence
    int lo, hi;  // positions [lo, hi) seen by any row of the tile
    int t0, nt;  // key tiles t0 .. t0 + nt - 1 (nt >= 1: an item that sees nothing still writes its zeros)
};

template <int ROWS, int KEYS>
__device__ __forceinline__ Item item_of(const AttnArgs &a, const Seq &s, int rt) {
    Item it;
    const int rows = s.qn * a.group;
    it.nrt = (rows + ROWS - 1) / ROWS;
    const int r0 = rt * ROWS, r1 = min(r0 + ROWS, rows) - 1;
    const int p0 = s.kv - s.qn + r0 / a.group, p1 = s.kv - s.qn + r1 / a.group;
    it.hi = a.causal ? min(max(p1 + 1, 0), s.kv) : s.kv;
    it.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), it.hi) : 0;
    it.t0 = it.lo / KEYS;
    it.nt = max((it.hi + KEYS - 1) / KEYS - it.t0, 1);
    return it;
}

// Units of one key/value head of sequence s, summed by one thread or (WARP) by a warp.
template <int ROWS, int KEYS, bool WARP>
__device__ __forceinline__ long long head_units(const AttnArgs &a, const Seq &s) {
    const int nrt = (s.qn * a.group + ROWS - 1) / ROWS;
    long long n = 0;
    for (int rt = WARP ? (int)(threadIdx.x & 31) : 0; rt < nrt; rt += WARP ? 32 : 1) n += item_of<ROWS, KEYS>(a, s, rt).nt;
    if (WARP) {
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(~0u, n, o);
    }
    return n;
}

// Where a CTA's range begins, and how many units it has.
struct Plan {
    long long total;  // units of the whole call
    long long first, count;
    int b, head, rt, tile;  // first unit: sequence, head, row tile, key tile within the item
    int ctas;               // CTAs that have units
};

struct PlanShared {
    long long sums[32];
    Plan plan;
};

__device__ __forceinline__ long long range_start(long long total, int c, int ctas) { return total * c / ctas; }
__device__ __forceinline__ int range_owner(long long total, long long unit, int ctas) {
    return (int)(((unit + 1) * ctas - 1) / total);
}

// Called by all THREADS threads of the CTA.  Workers (threads, or warps where
// sequences have many row tiles) sum contiguous runs of sequences; a scan
// over the workers finds the run that holds the CTA's first unit, and its
// worker walks down to the sequence, head, row tile and key tile.
template <int ROWS, int KEYS, int THREADS, int MIN_UNITS, bool WARP>
__device__ __forceinline__ void make_plan_by(const AttnArgs &a, PlanShared &sh) {
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int worker = WARP ? warp : (int)threadIdx.x, workers = WARP ? W : THREADS;
    const int per = (a.b.batch + workers - 1) / workers;
    const int b0 = min(worker * per, a.b.batch), b1 = min(b0 + per, a.b.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_units<ROWS, KEYS, WARP>(a, load_seq(a.b, b)) * a.kv_heads;
    long long before = 0;  // units of the workers before this one in its warp
    long long warp_sum = mine;
    if (!WARP) {
        long long inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += v;
        }
        before = inc - mine;
        warp_sum = __shfl_sync(~0u, inc, 31);
    }
    if (lane == 0) sh.sums[warp] = warp_sum;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const long long v = sh.sums[i];
        if (i < warp) before += v;
        total += v;
    }
    int ctas = (int)gridDim.x;
    if (total < (long long)ctas * MIN_UNITS) ctas = max((int)((total + MIN_UNITS - 1) / MIN_UNITS), 1);
    const int c = (int)blockIdx.x;
    const long long first = c < ctas ? range_start(total, c, ctas) : total;
    const long long last = c < ctas ? range_start(total, c + 1, ctas) : total;
    if (first < last && first >= before && first < before + mine) {
        long long res = first - before;
        int b = b0;
        for (;; ++b) {
            const Seq s = load_seq(a.b, b);
            const long long n = head_units<ROWS, KEYS, WARP>(a, s);
            if (res < n * a.kv_heads) {
                const int head = (int)(res / n);
                res -= head * n;
                int rt = 0;
                if (WARP) {  // 32 row tiles at a time
                    const int nrt = (s.qn * a.group + ROWS - 1) / ROWS;
                    for (;; rt += 32) {
                        const int v = rt + lane < nrt ? item_of<ROWS, KEYS>(a, s, rt + lane).nt : 0;
                        long long inc = v;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const long long x = __shfl_up_sync(~0u, inc, o);
                            if (lane >= o) inc += x;
                        }
                        const unsigned m = __ballot_sync(~0u, inc > res);
                        if (m) {
                            const int k = __ffs(m) - 1;
                            res -= __shfl_sync(~0u, inc - v, k);
                            rt += k;
                            break;
                        }
                        res -= __shfl_sync(~0u, inc, 31);
                    }
                } else {
                    for (;; ++rt) {
                        const int v = item_of<ROWS, KEYS>(a, s, rt).nt;
                        if (res < v) break;
                        res -= v;
                    }
                }
                if (!WARP || lane == 0) {
                    sh.plan.b = b;
                    sh.plan.head = head;
                    sh.plan.rt = rt;
                    sh.plan.tile = (int)res;
                }
                break;
            }
            res -= n * a.kv_heads;
        }
    }
    if (threadIdx.x == 0) {
        sh.plan.total = total;
        sh.plan.first = first;
        sh.plan.count = last - first;
        sh.plan.ctas = ctas;
    }
    __syncthreads();
}

template <int ROWS, int KEYS, int THREADS, int MIN_UNITS>
__device__ __forceinline__ void make_plan(const AttnArgs &a, PlanShared &sh) {
    if (a.few_tiles)
        make_plan_by<ROWS, KEYS, THREADS, MIN_UNITS, false>(a, sh);
    else
        make_plan_by<ROWS, KEYS, THREADS, MIN_UNITS, true>(a, sh);
}

// Walks a CTA's range piece by piece (a piece: its units of one item).
template <int ROWS, int KEYS>
struct Pieces {
    const AttnArgs &a;
    long long left;  // units not yet handed out
    long long at;    // index of the next unit
    int b, head, rt, tile;
    Seq s;
    // the piece
    Item it;
    int n;              // key tiles it.t0 + tile0 .. of the piece
    int tile0;          // first of them, within the item
    bool begins, ends;  // it holds the item's first and last tile

    __device__ __forceinline__ Pieces(const AttnArgs &args, const Plan &p)
        : a(args), left(p.count), at(p.first), b(p.b), head(p.head), rt(p.rt), tile(p.tile) {
        if (left > 0) s = load_seq(a.b, b);
    }

    __device__ __forceinline__ bool next() {
        if (left <= 0) return false;
        while (rt * ROWS >= s.qn * a.group) {  // past the sequence's row tiles
            rt = 0;
            if (s.qn == 0 || ++head == a.kv_heads) {
                head = 0;
                s = load_seq(a.b, ++b);
            }
        }
        it = item_of<ROWS, KEYS>(a, s, rt);
        tile0 = tile;
        n = (int)min((long long)(it.nt - tile), left);
        begins = tile == 0;
        ends = tile + n == it.nt;
        left -= n;
        at += n;
        tile = 0;
        ++rt;
        return true;
    }
    __device__ __forceinline__ int row0() const { return (rt - 1) * ROWS; }
    __device__ __forceinline__ int rows() const { return min(ROWS, s.qn * a.group - row0()); }
    // Partial-result slot of a piece that is not a whole item.
    __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (begins ? 1 : 0); }
    // CTAs that share the item of a piece that begins but does not end it.
    __device__ __forceinline__ int parts(const Plan &p) const {
        return range_owner(p.total, at - n + it.nt - 1, p.ctas) - (int)blockIdx.x + 1;
    }
};

// Tensor-map coordinates of the copy of positions p .. p + box_rows - 1 (one
// page holds them): the page, or num_pages, from which copies read zeros,
// for one that the item does not see or the cache does not have.
__device__ __forceinline__ int page_of(const AttnArgs &a, int b, int p, int lo, int hi) {
    if (p >= hi || p + a.box_rows <= lo) return a.num_pages;
    const int page = __ldg(a.b.table + (long long)b * a.b.table_stride + p / a.page_size);
    if ((unsigned)page < (unsigned)a.num_pages) return page;
    atomicExch(&g_bad_index, 1);
    return a.num_pages;
}

// 4-D tensor copy global -> shared, completion counted on `bar`.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace w4a16
