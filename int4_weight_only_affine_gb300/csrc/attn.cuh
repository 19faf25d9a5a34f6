// How f16_attention shares its work out, common to its kernels.
//
// The query rows of one sequence and key/value head are its new tokens times
// the head's query heads: row r is token r / G of the sequence, query head
// r % G of the group (G = q_heads / kv_heads).  An item is a tile of `rows`
// such rows (of one sequence, one key/value head) with the range of
// positions [lo, hi) that any of its rows sees; a unit is one tile of `keys`
// positions of that range.  An item costs its units (twice, if it has many
// rows) and, for its queries and outputs, EXTRA more.  All items' costs, in
// the order (sequence, head, row tile, key tile), are cut into one contiguous
// range per CTA, equal to within a unit, whatever the lengths; cuts near an
// item's end are moved to it; where the items are few and alike each goes
// whole to one CTA, and where they are many and none costs more than an even
// share they are taken whole from a queue (Cut, make_plan_by).  An item cut by
// a range boundary is computed in parts: each part's CTA leaves its
// unnormalised output, running maximum and sum in the workspace and counts
// itself in; when a CTA is done with its own range it waits for the parts of the items it shares and joins
// its share of their rows, in the parts' order.  A CTA waits only if every CTA
// of the launch had begun whenever it counted a part in (so each will finish,
// whatever else the GPU runs); otherwise it says so as it counts, and the last
// to count a part of the item in joins all of it (join_rule.h).  (A cooperative launch would
// promise the same, but is not overlapped with the end of the kernel before:
// 2.6 us a call.)  Every CTA works its range out from the lengths by itself:
// the host needs no lengths, and no result depends on which CTA computes it, so
// results repeat.
#pragma once

#include <math.h>

#include "join_rule.h"
#include "kv.cuh"

namespace w4a16 {

struct AttnArgs {
    KvBatch b;
    const uint16_t *q;
    uint16_t *y;
    float *lse;
    long long q_token, q_head, y_token, y_head;
    FastDiv group, page_size;
    int kv_heads, head_dim;
    int causal, window;
    int num_pages, box_rows;
    int few_tiles;  // a sequence is expected to have few row tiles (chooses how the plan is summed)
    int may_queue;  // there may be more items than CTAs, of sequences with many row tiles
    float scale;    // times log2(e): the softmax is taken in powers of two
    float *part_o;  // [2 * grid][rows x head_dim], in the order of the kernel that writes it
    float *part_ml; // [2 * grid][rows][2]: running maximum (base-2 scaled scores) and sum
    // Of the item that starts in a CTA's range, zero between calls: parts
    // counted in (and above bit 16 those that will not wait), and CTAs done
    // with it.
    unsigned *arrived, *left;
    unsigned *begun, *begun_before;  // CTAs begun in all calls, and in the calls before
    unsigned *taken, *finished;      // of a queue of items: those taken, CTAs that found it empty (zero between calls)
};

// A CTA's part of an item that several CTAs share.
struct Part {
    int first, parts, index;  // CTA whose range the item starts in, CTAs that share it, this one's place among them
    int q0, head, row0, rows;  // the sequence's first token, key/value head, rows of the item
};

// How a kernel's work is cut: rows and positions of a unit, an item's extra
// cost, the least cost worth a CTA of its own.  A unit of an item of more than
// FEW_ROWS rows costs 2.  Joining an item's parts takes as long as some units:
//  * Where there are no more items than CTAs and none costs more than an even
//    share and SLACK, each is left whole (single tokens of 16 sequences of 300
//    positions, 8 heads of 128: 8.7 us, against 16.1 cut into even shares; of
//    64 sequences of 2000, 2 heads: 29, against 38; items of 300 positions and
//    32 rows: 13.4, against 22).
//  * Else the two key tiles next to an end of an item that costs no more than
//    that are not cut off (single tokens of 24 sequences of 300: 13, against
//    18); of a costlier one, which is cut all the same, LONG (few rows) or two
//    (many).  With an even share of 7, a 16001-position item of 128 rows
//    takes 26 us with LONG = 0, 28 with 1; 600 positions of heads of 256 with
//    4 rows 16.9 with 0, 14.2 with 1.
// QUEUE: where there are more items than CTAs, none much above an even share,
// no item need be cut (prompt of 8192 tokens, 16 heads of 128 on 8: 222 us,
// against 229 in ranges; two of 1000, 32 heads on 8: 37, against 43; of 2048:
// 53, against 57).
template <int ROWS_, int KEYS_, int EXTRA_, int LEAST_, int FEW_ROWS_, int SLACK_, int LONG_, bool QUEUE_>
struct Cut {
    static constexpr int ROWS = ROWS_, KEYS = KEYS_, EXTRA = EXTRA_, LEAST = LEAST_, FEW_ROWS = FEW_ROWS_, SLACK = SLACK_, LONG = LONG_;
    static constexpr bool QUEUE = QUEUE_;
};

struct Item {
    int rows;    // of the tile
    int lo, hi;  // positions [lo, hi) seen by any row of the tile
    int t0, nt;  // key tiles t0 .. t0 + nt - 1 (nt >= 1: an item that sees nothing still writes its zeros)
    int weight;  // of a unit
};

template <class C>
__device__ __forceinline__ Item item_of(const AttnArgs &a, const Seq &s, int rt) {
    constexpr int ROWS = C::ROWS, KEYS = C::KEYS;
    Item it;
    const int rows = s.qn * (int)a.group.d;
    const int r0 = rt * ROWS, r1 = min(r0 + ROWS, rows) - 1;
    it.rows = r1 - r0 + 1;
    const int p0 = s.kv - s.qn + r0 / a.group, p1 = s.kv - s.qn + r1 / a.group;
    it.hi = a.causal ? min(max(p1 + 1, 0), s.kv) : s.kv;
    it.lo = a.window > 0 ? min(max(p0 - a.window + 1, 0), it.hi) : 0;
    it.t0 = it.lo / KEYS;
    it.nt = max((it.hi + KEYS - 1) / KEYS - it.t0, 1);
    it.weight = it.rows > C::FEW_ROWS ? 2 : 1;
    return it;
}

// Cost of one key/value head of sequence s, summed by one thread or (WARP) by a warp.
template <class C>
__device__ __forceinline__ int cost_of(const Item &it) {
    return it.nt * it.weight + C::EXTRA;
}
template <class C>
__device__ __forceinline__ int row_tiles(const AttnArgs &a, const Seq &s) {
    return (s.qn * (int)a.group.d + C::ROWS - 1) / C::ROWS;
}
// (And into most, if that is less, the cost of its costliest item.)
template <class C, bool WARP>
__device__ __forceinline__ uint32_t head_cost(const AttnArgs &a, const Seq &s, uint32_t &most) {
    const int nrt = row_tiles<C>(a, s);
    uint32_t n = 0;
    for (int rt = WARP ? (int)(threadIdx.x & 31) : 0; rt < nrt; rt += WARP ? 32 : 1) {
        const uint32_t cost = cost_of<C>(item_of<C>(a, s, rt));
        n += cost;
        most = max(most, cost);
    }
    return WARP ? __reduce_add_sync(~0u, n) : n;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Where a CTA's range begins, and its length.  The first `more` CTAs' ranges
// are per + 1 long, the others' per.  (Calls whose cost may reach 2^31 are
// refused on the host.)
struct Plan {
    uint32_t per, more;
    uint32_t first, count;
    int b, head, rt, off;  // its first item: sequence, head, row tile; how far into the item's cost it begins
    uint32_t queue;  // if not 0: no ranges, but a queue of so many places (Queue)
};

// The CTA whose range holds a unit of cost.
__device__ __forceinline__ uint32_t owner(const Plan &p, uint32_t at) {
    const uint32_t cut = p.more * (p.per + 1);
    return at < cut ? at / (p.per + 1) : p.more + (at - cut) / p.per;
}

constexpr uint32_t kDisorder = 0xFFFFFFFFu;  // in place of the greatest cost: offsets out of order

struct PlanShared {
    uint32_t sums[32], items[32], most[32], tiles[32];
    Plan plan;
    unsigned begun_before;
};

// Called by all THREADS threads of the CTA.  Workers (threads, or warps where
// sequences have many row tiles) sum contiguous runs of sequences; a scan
// over the workers finds the run that holds the beginning of the CTA's range,
// and its worker walks down to the sequence, head and row tile.
template <class C, int THREADS, bool WARP>
__device__ __forceinline__ void make_plan_by(const AttnArgs &a, PlanShared &sh) {
    constexpr uint32_t W = THREADS / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t worker = WARP ? warp : threadIdx.x, workers = WARP ? W : THREADS;
    const uint32_t batch = (uint32_t)a.b.batch, per = (batch + workers - 1) / workers;
    const uint32_t b0 = min(worker * per, batch), b1 = min(b0 + per, batch);
    uint32_t mine = 0, items = 0, most = 0, tiles = 0, cost = 0;  // cost: of a head of the worker's last sequence
    Seq s = {0, 0, 0, true, true};
    for (uint32_t b = b0; b < b1; ++b) {
        s = load_seq(a.b, (int)b);
        cost = head_cost<C, WARP>(a, s, most);
        mine += cost * a.kv_heads;
        const uint32_t n = row_tiles<C>(a, s);
        items += n * a.kv_heads;
        tiles = max(tiles, n);
        if (!s.ordered) most = kDisorder;
    }
    uint32_t before = 0, warp_sum = mine;  // cost of earlier workers
    if (!WARP) {
        const uint32_t inc = warp_scan(mine, lane);
        before = inc - mine;
        warp_sum = __shfl_sync(~0u, inc, 31);
    }
    if (C::QUEUE && WARP) {
        tiles = __reduce_max_sync(~0u, tiles);
        if (lane == 0) sh.tiles[warp] = tiles;
    }
    const uint32_t warp_items = WARP ? items : __reduce_add_sync(~0u, items), warp_most = __reduce_max_sync(~0u, most);
    if (lane == 0) {
        sh.sums[warp] = warp_sum;
        sh.items[warp] = warp_items;
        sh.most[warp] = warp_most;
    }
    __syncthreads();
    uint32_t total = 0, all_items = 0, all_most = 0, all_tiles = 0, items_before = 0;
#pragma unroll
    for (uint32_t i = 0; i < W; ++i) {
        const uint32_t v = sh.sums[i], n = sh.items[i];
        if (i < warp) {
            before += v;
            items_before += n;
        }
        total += v;
        all_items += n;
        all_most = max(all_most, sh.most[i]);
        if (C::QUEUE && WARP) all_tiles = max(all_tiles, sh.tiles[i]);
    }
    uint32_t ctas = gridDim.x;
    const uint32_t c = blockIdx.x;
    if (total < ctas * C::LEAST) ctas = max((total + C::LEAST - 1) / C::LEAST, 1u);
    Plan p;
    p.per = total / ctas;
    p.more = total - p.per * ctas;
    p.first = p.per * c + min(c, p.more);
    p.count = c < ctas ? p.per + (c < p.more ? 1 : 0) : 0;
    p.queue = 0;
    if (C::QUEUE && WARP && all_items > gridDim.x && all_most <= p.per + C::SLACK) {
        // Taken whole, costliest first, items of at most an even share and SLACK
        // end at about the same time, if their costs differ or about fill the rounds.
        const unsigned long long places = (unsigned long long)all_tiles * a.kv_heads * batch, n = all_items;
        const uint32_t rounds = (all_items + gridDim.x - 1) / gridDim.x;
        if (places <= 2 * n && (4ull * total <= 3 * n * all_most || (unsigned long long)rounds * total <= n * (p.per + C::SLACK / 2)))
            p.queue = (uint32_t)places;
    }
    auto publish = [&] {
        sh.plan = p;
        // The pages of the first tile will be wanted next.
        const Item it = item_of<C>(a, s, p.rt);
        const int at = (it.t0 + max(p.off - C::EXTRA, 0) / it.weight) * C::KEYS;
        if (at < it.hi)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.b.table + (long long)p.b * a.b.table_stride + at / a.page_size));
    };
    if (all_most == kDisorder) {  // (reported by load_seq) no sum above is to be relied on: nothing is computed
        p.count = 0;
    } else if (C::QUEUE && WARP && p.queue) {
        p.count = 0;
    } else if (all_items <= gridDim.x && all_most <= p.per + C::SLACK) {  // an item to a CTA
        p.count = c < all_items ? 1 : 0;
        if (!WARP) items_before += warp_scan(items, lane) - items;
        if (c >= items_before && c - items_before < items) {
            uint32_t res = c - items_before, b = b0, nrt;
            for (;; ++b) {
                s = load_seq(a.b, (int)b);
                nrt = row_tiles<C>(a, s);
                if (res < nrt * a.kv_heads) break;
                res -= nrt * a.kv_heads;
            }
            p.b = (int)b;
            p.head = (int)(res / nrt);
            p.rt = (int)(res - p.head * nrt);
            p.off = 0;
            p.count = cost_of<C>(item_of<C>(a, s, p.rt));
            if (!WARP || lane == 0) publish();
        }
    } else if (p.count > 0 && p.first >= before && p.first - before < mine) {
        uint32_t res = p.first - before;
        uint32_t b = b0;
        if (b1 - b0 > 1)
            for (;; ++b) {
                s = load_seq(a.b, (int)b);
                cost = head_cost<C, WARP>(a, s, most);
                if (res < cost * a.kv_heads) break;
                res -= cost * a.kv_heads;
            }
        p.b = (int)b;
        p.head = (int)(res / cost);
        res -= p.head * cost;
        int rt = 0;
        if (WARP) {  // 32 row tiles at a time
            const int nrt = row_tiles<C>(a, s);
            for (;; rt += 32) {
                const uint32_t v = rt + lane < nrt ? cost_of<C>(item_of<C>(a, s, rt + lane)) : 0;
                const uint32_t inc = warp_scan(v, lane);
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
                const uint32_t v = cost_of<C>(item_of<C>(a, s, rt));
                if (res < v) break;
                res -= v;
            }
        }
        p.rt = rt;
        p.off = (int)res;
        if (!WARP || lane == 0) publish();
    }
    if (p.count == 0 && threadIdx.x == 0) sh.plan = p;
    __syncthreads();
}

template <class C, int THREADS>
__device__ __forceinline__ void make_plan(const AttnArgs &a, PlanShared &sh) {
    if (!C::QUEUE && a.few_tiles)  // (a queue is for many)
        make_plan_by<C, THREADS, false>(a, sh);
    else
        make_plan_by<C, THREADS, true>(a, sh);
}

// Walks a CTA's range piece by piece (a piece: its key tiles of one item).
template <class C>
struct Pieces {
    static constexpr int ROWS = C::ROWS;
    const AttnArgs &a;
    uint32_t left;  // of the range's cost
    uint32_t at;    // cost before the next item
    int b, head, rt, off;
    int per;
    Seq s;
    // the piece
    Item it;
    int n;              // key tiles it.t0 + tile0 .. of the piece, one at least
    int tile0;          // first of them, within the item
    bool begins, ends;  // it holds the item's first and last tile

    __device__ __forceinline__ Pieces(const AttnArgs &args, const Plan &p)
        : a(args), left(p.count), at(p.first - p.off), b(p.b), head(p.head), rt(p.rt), off(p.off), per((int)p.per) {
        if (left > 0) s = load_seq(a.b, b);
    }

    // Cuts at key tile uncut_lo() or before are moved to the item's beginning,
    // at uncut_hi() or after to its end.
    __device__ __forceinline__ int snap() const {
        return cost_of<C>(it) > per + C::SLACK ? min(it.weight > 1 ? 2 : C::LONG, per / 3) : 2;
    }
    __device__ __forceinline__ int uncut_lo() const { return min(snap(), it.nt / 2); }
    __device__ __forceinline__ int uncut_hi() const { return max(it.nt - snap(), it.nt / 2 + 1); }
    // The key tile that a cut at cost x of the item comes before.
    __device__ __forceinline__ int cut_tile(int x) const {
        const int cut = x <= C::EXTRA ? 0 : (it.weight > 1 ? (x - C::EXTRA) >> 1 : x - C::EXTRA);
        return cut <= uncut_lo() ? 0 : (cut >= uncut_hi() ? it.nt : cut);
    }

    __device__ __forceinline__ bool next() {
        while (left > 0) {
            while (rt * ROWS >= s.qn * (int)a.group.d) {  // past the sequence's row tiles
                rt = 0;
                if (s.qn == 0 || ++head == a.kv_heads) {
                    head = 0;
                    s = load_seq(a.b, ++b);
                }
            }
            it = item_of<C>(a, s, rt);
            const int cost = cost_of<C>(it), end = (int)min((uint32_t)cost, left + off);
            tile0 = cut_tile(off);
            n = cut_tile(end) - tile0;
            begins = tile0 == 0;
            ends = tile0 + n == it.nt;
            left -= end - off;
            at += cost;
            off = 0;
            ++rt;
            if (n > 0) return true;  // else another CTA has all that this one might have of the item
        }
        return false;
    }
    __device__ __forceinline__ int row0() const { return (rt - 1) * ROWS; }
    __device__ __forceinline__ int rows() const { return it.rows; }
    // Partial-result slot of a piece that is not a whole item.
    __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (begins ? 1 : 0); }
    // Of a piece that is not a whole item.
    __device__ __forceinline__ Part part(const Plan &p) const {
        const uint32_t tiles0 = at - it.nt * it.weight;  // cost before the item's first tile
        const int first = begins ? (int)blockIdx.x : (int)owner(p, tiles0 + (uncut_lo() + 1) * it.weight - 1);
        const int last = ends ? (int)blockIdx.x : (int)owner(p, tiles0 + uncut_hi() * it.weight - 1);
        return Part{first, last - first + 1, (int)blockIdx.x - first, s.q0, head, row0(), rows()};
    }
};

// mbar_wait without a call, and without a look at the clock (which takes as
// long as most waits here) until the wait has become long.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    uint64_t t0 = 0;
    for (uint32_t spin = 0; spin < kMaxSpins; ++spin) {
        if (mbar_try(bar, parity)) return true;
        if ((spin & 63) == 63) {
            if (abort && *abort) return false;
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitNs) break;
        }
    }
    atomicExch(&g_wait_expired, 1);
    if (abort) *abort = 1;
    return false;
}

// The tensor maps' descriptors, fetched ahead of their first copies.
__device__ __forceinline__ void prefetch_maps(const CUtensorMap *k, const CUtensorMap *v) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(v) : "memory");
}

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

// 5-D tensor copy global -> shared, completion counted on `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
        "[%7];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

// Copies and MMAs take their operands from uniform registers.  Loops that
// issue them run on values of the whole warp (uniform), known as such to the
// compiler, with one elected thread issuing: lanes that each issue their own
// are run one after the other, at some 80 cycles a copy.
__device__ __forceinline__ bool elect_one() {  // the same thread of the (converged) warp each time
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
template <class T>
__device__ __forceinline__ T uniform(T v) {
    return __shfl_sync(~0u, v, 0);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^(a - b) for maxima of which either may be -infinity (nothing seen yet).
__device__ __forceinline__ float corr(float a, float b) { return a == -INFINITY ? 0.f : exp2_approx(a - b); }

// 1 / sum, 0 for a row that saw nothing; not finite if the sum is not.
__device__ __forceinline__ float inverse(float sum) { return sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum); }

// Natural logarithm of sum * 2^mx.
__device__ __forceinline__ float log_sum(float mx, float sum) {
    return sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
}

// Slot of part i of the item that starts in the range of CTA c: the beginning
// lies in the odd slot of c, every later part in the even slot of the next ones.
__device__ __forceinline__ long long part_slot(int c, int i) { return 2 * (c + i) + (i == 0 ? 1 : 0); }

// A CTA begins: by one thread, after the kernel before is done.  begun counts
// on from call to call; begun_before is moved up by the last CTA to begin,
// when every other has read it.
struct Begin {
    unsigned before, mine;
};
__device__ __forceinline__ Begin cta_begins(const AttnArgs &a) {
    Begin b;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(b.before) : "l"(a.begun_before) : "memory");
    b.mine = atomicAdd(a.begun, 1u);
    return b;
}
__device__ __forceinline__ void cta_has_begun(const AttnArgs &a, const Begin &b) {  // (when the count is back)
    if (b.mine + 1 == b.before + gridDim.x) *a.begun_before = b.before + gridDim.x;
}

// Counts a part in, by a thread that its writers have synchronised with;
// returns the item's count with it, and clears `waits` where the CTA may not
// wait for the others.  COPIED: the parts are read by copies.
template <bool COPIED>
__device__ __forceinline__ unsigned count_part(const AttnArgs &a, const Part &p, unsigned begun_before, bool &waits) {
    unsigned begun;  // (on its way while the fence is)
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(begun) : "l"(a.begun) : "memory");
    __threadfence();
    if (COPIED) asm volatile("fence.proxy.async.global;" ::: "memory");
    const unsigned mine = part_mark(begun == begun_before + gridDim.x, waits);
    return atomicAdd(a.arrived + p.first, mine) + mine;
}

// What this CTA joins (join_mode), asked by one thread with the count as it
// saw it; with `waits` it waits until all `parts` arrivals are in.  A wait is
// bounded: when it runs out, and where there are more arrivals than parts,
// w4a16_device_status says so.
__device__ __forceinline__ int await_parts(const AttnArgs &a, const Part &p, unsigned seen, bool waits, unsigned parts) {
    unsigned now = seen;
    if (waits)  // (the first look does not need `seen`, which may still be on its way)
        now = await_count(parts, kWaitNs, [&] {
            unsigned v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.arrived + p.first) : "memory");
            return v;
        }, [] { return global_ns(); });
    bool failed;
    const int mode = join_mode(now, seen, waits, parts, failed);
    if (failed) atomicExch(&g_wait_expired, 1);
    if (!waits && mode != kJoinNothing) __threadfence();
    return mode;
}

// A CTA is done with an item: the last of them all leaves its counts at zero.
__device__ __forceinline__ void part_done(const AttnArgs &a, const Part &p) {
    if (atomicAdd(a.left + p.first, 1u) == (unsigned)p.parts - 1) {
        a.arrived[p.first] = 0;
        a.left[p.first] = 0;
    }
}

// Launch as a programmatic dependent (the kernels wait for the one before
// first: it only takes the launch itself off the path).
template <class K>
int launch_dependent(K kernel, int grid, int threads, size_t smem, cudaStream_t stream, const CUtensorMap &mk,
                     const CUtensorMap &mv, const AttnArgs &a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, mk, mv, a) != cudaSuccess) {
        cudaGetLastError();
        return W4_ERR_LAUNCH;
    }
    return W4A16_OK;
}

}  // namespace w4a16
