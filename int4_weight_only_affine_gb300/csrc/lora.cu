// f16_lora: low-rank adapters of many requests beside a shared projection,
//     out[m] = y[m] + s_a (x[m] A_a^T) B_a^T,   a = ids[m]  (negative: out = y).
// The columns may be cut into slices (q | k | v, gate | up) with an A each: B's
// rows of a slice multiply that slice's h = x A^T.
//
// What bounds it: y is read and out written once, x read once, each adapter in
// use read once; the products (2 r flops an element of x and of y) are small
// beside that up to ranks of about 64.  So the rows of one adapter are gathered,
// h stays on the chip, and one launch does everything:
//  * A cluster of 8 CTAs takes a unit: up to `tile` rows of one adapter, and all or
//    one of several parts of the columns.  Its CTAs split K for h (shrink), add
//    their partial sums through distributed shared memory, and split the columns
//    for the second product (expand), so nothing passes through memory and no CTA
//    waits for one outside its cluster.  Parts of one item each make h
//    themselves: A comes from L2 then, and h is far less work than the columns.
//  * Which rows belong to which adapter is found by every CTA itself, for a scope
//    of up to 1024 rows: a histogram of ids in shared memory, a prefix sum
//    over the adapters, and the rows of the unit in order by a second one.  Any
//    mix of ids is served.  The CTAs of a cluster read an eighth of the ids each and
//    take the rest from one another, so that they agree on their units, and meet at
//    the same cluster barriers, even if another stream wrote ids meanwhile.
//  * Both products are mma.sync m16n8k16 with operands loaded straight from global
//    memory in fragment order: the order of k inside a product is free, so lane t
//    of a quad takes 16 contiguous bytes of a row and treats them as the k indexes
//    of two products.  With ranks of 16 to 64 a tcgen05 tile would be filled to an
//    eighth and h would have to go to shared memory in its layout; the bytes are
//    the bound, not the tensor rate.
//  * expand holds B's fragments of 32 columns in registers over all row tiles of the
//    unit.  The order of columns inside the four products is chosen so that a lane
//    holds 8 neighbouring ones of two rows: 16-byte loads of y and stores of out.
// Numerics: x and A are binary16, h and the sums fp32 (K in a fixed order).  h is
// multiplied by s_a, scaled by a power of two to the row's largest in
// [2^12, 2^13), and split into two binary16 numbers hi + lo: the second product
// then sees h to 2^-22 of the row's largest instead of 2^-11, for one product
// more.  y + delta is rounded once.
#include <cooperative_groups.h>

#include <mutex>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace w4a16 {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kCluster = 8;
constexpr int kScope = 1024;        // rows whose ids a CTA sorts
constexpr int kMaxAdapters = 4096;  // buckets of the histogram
constexpr int kMaxSlices = 4;
constexpr int kMaxRank = 128;
constexpr int kColBlock = 32;  // columns of a warp's step

struct LoraArgs {
    const uint16_t *x, *y, *a, *b;
    uint16_t *out;
    const float *scale;
    const int32_t *ids;
    long long x_row, y_row, out_row, a_adapter, b_adapter;
    int M, K, N, adapters, rank, slices;
    int col[kMaxSlices + 1];    // first column of each slice, N at the end
    int block[kMaxSlices + 1];  // column blocks before each slice
    int scope, clusters;        // rows of a scope, clusters to a scope
    int tile;                   // rows of a unit: 16, 32 or 64
    int parts;                  // most parts of an item's columns
    int copy;                   // out is not y: rows without an adapter are copied
    uint32_t off_red, off_hist;  // byte offsets in shared memory (h at 0)
};

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }

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

// Shrink: partial sums over the CTA's share of K of h[row][slice][r], for the
// unit's n rows, into h[row][R] (R = slices * RK; ranks past `rank` get zero).
template <int RK>
__device__ __forceinline__ void shrink(const LoraArgs &p, const uint16_t *a, const int *rows, int n, int crank,
                                       float *h, float *red) {
    constexpr int MT = RK >= 64 ? 4 : RK / 16;       // 16-rank tiles that a warp holds at a time
    constexpr int G = 16 * MT;                       // ranks of a pass
    constexpr int kAhead = RK >= 64 ? 1 : RK == 32 ? 2 : 4;  // 32-k blocks loaded ahead
    const int R = p.slices * RK;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rgroups = n <= 16 ? 1 : n <= 32 ? 2 : 4;  // of 16 rows
    const int kgroups = kWarps / rgroups;
    const int rg = warp % rgroups, kg = warp / rgroups;
    const int nrows = 16 * rgroups;
    const int kb = (p.K + 31) / 32;
    const int share0 = (int)((long long)kb * crank / kCluster), share1 = (int)((long long)kb * (crank + 1) / kCluster);
    const int k0 = share0 + (share1 - share0) * kg / kgroups, k1 = share0 + (share1 - share0) * (kg + 1) / kgroups;
    const uint16_t *xr[2];
    bool xv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = rg * 16 + 8 * i + g;
        xv[i] = r < n;
        xr[i] = p.x + (xv[i] ? rows[r] : rows[0]) * p.x_row + 8 * t;
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int pass = 0; pass < R / G; ++pass) {
        float acc[MT][2][4] = {};
        const uint16_t *ar[2 * MT];
        bool av[2 * MT];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int pr = pass * G + 8 * i + g, s = pr / RK, r = pr % RK;
            av[i] = r < p.rank;
            ar[i] = a + ((long long)s * p.rank + (av[i] ? r : 0)) * p.K + 8 * t;
        }
        for (int b = k0; b < k1; b += kAhead) {
            uint4 av4[kAhead][2 * MT], xv4[kAhead][2];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const bool in = b + q < k1 && 32 * (b + q) + 8 * t < p.K;
#pragma unroll
                for (int i = 0; i < 2; ++i) xv4[q][i] = in && xv[i] ? load16(xr[i] + 32 * (b + q)) : zero;
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) av4[q][i] = in && av[i] ? load16(ar[i] + 32 * (b + q)) : zero;
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 u = av4[q][2 * m], l = av4[q][2 * m + 1];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        mma_16816(acc[m][i], u.x, l.x, u.y, l.y, xv4[q][i].x, xv4[q][i].y);
                        mma_16816(acc[m][i], u.z, l.z, u.w, l.w, xv4[q][i].z, xv4[q][i].w);
                    }
                }
        }
        // red [kgroups][nrows][G]
        float *mine = red + (kg * nrows + rg * 16) * G;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[(8 * i + 2 * t + (e & 1)) * G + 16 * m + g + 8 * (e >> 1)] = acc[m][i][e];
        __syncthreads();
        for (int e = threadIdx.x; e < n * G; e += kThreads) {
            float v = 0.f;
            for (int q = 0; q < kgroups; ++q) v += red[q * nrows * G + e];
            h[e / G * R + pass * G + e % G] = v;
        }
        __syncthreads();
    }
}

// Place of ranks r, r + 1 (r even) of slice s of row `row` among the fragments of
// the second product: word index in frag[half][row tile][slice * RK / 16 + k16][lane][4].
template <int RK>
__device__ __forceinline__ int frag_word(int row, int s, int r) {
    const int g = row & 7, up = row >> 3 & 1;
    int t, k16, q;
    if (RK == 16) {  // lane t holds ranks 4t .. 4t + 3
        t = r >> 2;
        k16 = 0;
        q = r >> 1 & 1;
    } else {  // lane t holds ranks 8t .. 8t + 7 of 32
        t = r >> 3 & 3;
        k16 = 2 * (r >> 5) + (r >> 2 & 1);
        q = r >> 1 & 1;
    }
    return ((s * (RK / 16) + k16) * 32 + g * 4 + t) * 4 + up + 2 * q;
}

// Adds the cluster's partial sums of the rows that this CTA owns, scales and
// splits them, and leaves the fragments with every CTA of the cluster.
template <int RK>
__device__ __forceinline__ void exchange(const LoraArgs &p, float scale, int n, float *h, uint32_t *frag, float *inv,
                                         int crank) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA's sums are in place, and its fragments' room is free
    const int R = p.slices * RK, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half_words = p.tile / 16 * (R / 16) * 128;  // words of the hi (and of the lo) fragments
    for (int row = crank + kCluster * warp; row < n; row += kCluster * kWarps) {
        float2 v[kMaxSlices * RK / 64 > 0 ? kMaxSlices * RK / 64 : 1];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < kMaxSlices * RK / 64; ++j) {
            const int r = 64 * j + 2 * lane;
            v[j] = make_float2(0.f, 0.f);
            if (r < R) {
                float2 part[kCluster];
#pragma unroll
                for (int c = 0; c < kCluster; ++c)
                    part[c] = *reinterpret_cast<const float2 *>(cluster.map_shared_rank(h, c) + row * R + r);
#pragma unroll
                for (int c = 0; c < kCluster; ++c) {
                    v[j].x += part[c].x;
                    v[j].y += part[c].y;
                }
                const bool used = r % RK < p.rank;  // (the rank is even)
                v[j].x = used ? v[j].x * scale : 0.f;
                v[j].y = used ? v[j].y * scale : 0.f;
            }
            top = fmaxf(top, fmaxf(fabsf(v[j].x), fabsf(v[j].y)));
            if (!(fabsf(v[j].x) < __int_as_float(0x7F800000) && fabsf(v[j].y) < __int_as_float(0x7F800000)))
                top = __int_as_float(0x7F800000);  // (NaN too)
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // 2^(12 - e) for a largest value in [2^e, 2^(e + 1)); 1 for rows of zeros and those that are not finite.
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const int shift = e == 128 || top == 0.f ? 0 : 12 - max(e, -100);
        const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
        if (lane < kCluster) cluster.map_shared_rank(inv, lane)[row] = __uint_as_float((uint32_t)(127 - shift) << 23);
        const int base = row / 16 * (R / 16) * 128;
#pragma unroll
        for (int j = 0; j < kMaxSlices * RK / 64; ++j) {
            const int r = 64 * j + 2 * lane;
            if (r >= R) continue;
            const float a = v[j].x * up, b = v[j].y * up;
            const uint32_t hi = pack(a, b);
            const float2 f = unpack(hi);
            const float la = a - f.x, lb = b - f.y;
            const uint32_t lo = pack(fabsf(la) < 1e30f ? la : 0.f, fabsf(lb) < 1e30f ? lb : 0.f);
            const int w = base + frag_word<RK>(row & 15, r / RK, r % RK);
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                uint32_t *dst = cluster.map_shared_rank(frag, c);
                dst[w] = hi;
                dst[half_words + w] = lo;
            }
        }
    }
    cluster.sync();
}

// Expand: out = y + h B^T over the CTA's column blocks [b0, b1) of the unit's rows.
template <int RK>
__device__ __forceinline__ void expand(const LoraArgs &p, const uint16_t *bw, const int *rows, int n,
                                       const uint32_t *frag, const float *inv, int b0, int b1) {
    constexpr int KS = RK / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int R16 = p.slices * KS, tiles = (n + 15) / 16;
    const uint4 *fr = reinterpret_cast<const uint4 *>(frag);
    const int half = p.tile / 16 * R16 * 32;
    for (int blk = b0 + warp; blk < b1; blk += kWarps) {
        int s = 0;
        while (s + 1 < p.slices && blk >= p.block[s + 1]) ++s;
        const int c0 = p.col[s] + (blk - p.block[s]) * kColBlock, c1 = min(c0 + kColBlock, p.col[s + 1]);
        // Column (product j, n = g) is c0 + 8 (g / 2) + 2 j + g % 2.
        uint32_t bf[4][KS][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + 8 * (g >> 1) + 2 * j + (g & 1);
            const uint16_t *row = bw + (long long)c * p.rank;
            if (RK == 16) {
                uint2 v = make_uint2(0u, 0u);
                if (c < c1 && 4 * t < p.rank) v = __ldg(reinterpret_cast<const uint2 *>(row + 4 * t));
                bf[j][0][0] = v.x;
                bf[j][0][1] = v.y;
            } else {
#pragma unroll
                for (int q = 0; q < KS / 2; ++q) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (c < c1 && 32 * q + 8 * t < p.rank) v = load16(row + 32 * q + 8 * t);
                    bf[j][2 * q][0] = v.x;
                    bf[j][2 * q][1] = v.y;
                    bf[j][2 * q + 1][0] = v.z;
                    bf[j][2 * q + 1][1] = v.w;
                }
            }
        }
        const bool cv = c0 + 8 * t < c1;
        const int col = c0 + 8 * t;
        uint4 yv[2];
        auto fetch = [&](int tile, uint4(&v)[2]) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * tile + 8 * i + g;
                if (cv && r < n) v[i] = *reinterpret_cast<const uint4 *>(p.y + rows[r] * p.y_row + col);
            }
        };
        fetch(0, yv);
        for (int tile = 0; tile < tiles; ++tile) {
            uint4 next[2];
            if (tile + 1 < tiles) fetch(tile + 1, next);
            float d[4][4] = {};
            const uint4 *f = fr + (tile * R16 + s * KS) * 32 + lane;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint4 hi = f[k * 32], lo = f[half + k * 32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_16816(d[j], hi.x, hi.y, hi.z, hi.w, bf[j][k][0], bf[j][k][1]);
                    mma_16816(d[j], lo.x, lo.y, lo.z, lo.w, bf[j][k][0], bf[j][k][1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * tile + 8 * i + g;
                if (cv && r < n) {
                    const float f = inv[r];
                    const uint32_t w[4] = {yv[i].x, yv[i].y, yv[i].z, yv[i].w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 old = unpack(w[j]);
                        o[j] = pack(fmaf(d[j][2 * i], f, old.x), fmaf(d[j][2 * i + 1], f, old.y));
                    }
                    *reinterpret_cast<uint4 *>(p.out + rows[r] * p.out_row + col) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                yv[i] = next[i];
            }
        }
    }
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
__global__ void __launch_bounds__(kThreads, RK == 128 ? 1 : 2) lora_kernel(const __grid_constant__ LoraArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scratch[kWarps], rows[64], unit[3];
    __shared__ float inv[64];
    __shared__ __align__(16) int own[kScope / kCluster];  // buckets of this CTA's share of the rows, -1 past the scope
    cg::cluster_group cluster = cg::this_cluster();
    float *h = reinterpret_cast<float *>(smem);                   // [tile][R]
    float *red = reinterpret_cast<float *>(smem + p.off_red);     // partial sums of the warps, then the fragments
    uint32_t *frag = reinterpret_cast<uint32_t *>(red);
    int *hist = reinterpret_cast<int *>(smem + p.off_hist);       // rows of each adapter; of none at the end
    const int tid = threadIdx.x, crank = (int)(blockIdx.x % kCluster), cl = (int)(blockIdx.x / kCluster);
    const int scope = cl / p.clusters, q = cl % p.clusters;
    const int row0 = scope * p.scope, nrow = min(p.scope, p.M - row0);
    const int buckets = p.adapters + 1;
    for (int i = tid; i < buckets; i += kThreads) hist[i] = 0;
    pdl_wait();
    constexpr int kShare = kScope / kCluster;
    if (tid < kShare) {
        const int r = crank * kShare + tid;
        int bucket = -1;
        if (r < nrow) {
            const int v = __ldg(p.ids + row0 + r);
            if (v >= p.adapters) atomicExch(&g_bad_index, 1);
            bucket = v < 0 || v >= p.adapters ? p.adapters : v;
        }
        own[tid] = bucket;
    }
    cluster.sync();
    // Four rows a thread, in order.
    constexpr int kMine = kScope / kThreads;
    static_assert(kMine == 4 && kShare % kMine == 0, "a thread's rows come from one CTA in one read");
    const int4 four = *reinterpret_cast<const int4 *>(cluster.map_shared_rank(own, tid * kMine / kShare) + tid * kMine % kShare);
    const int id[kMine] = {four.x, four.y, four.z, four.w};
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        if (id[i] >= 0) atomicAdd(hist + id[i], 1);
    __syncthreads();
    // Items: up to `tile` rows of one bucket.  This thread's buckets are in a row.
    const int per = (buckets + kThreads - 1) / kThreads;
    int mine = 0, items;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < buckets && (b < p.adapters || p.copy)) mine += (hist[b] + p.tile - 1) / p.tile;
    }
    const int first = block_scan(mine, scratch, items);
    const int parts = max(1, min(p.parts, p.clusters / max(items, 1)));
    for (int u = q; u < items * parts; u += p.clusters) {
        const int item = u % items, part = u / items;
        if (item >= first && item < first + mine) {
            int at = first;
            for (int i = 0; i < per; ++i) {
                const int b = tid * per + i;
                if (b < buckets && (b < p.adapters || p.copy)) {
                    const int c = (hist[b] + p.tile - 1) / p.tile;
                    if (item >= at && item < at + c) {
                        unit[0] = b;
                        unit[1] = (item - at) * p.tile;
                        unit[2] = min(p.tile, hist[b] - (item - at) * p.tile);
                    }
                    at += c;
                }
            }
        }
        __syncthreads();
        const int bucket = unit[0], skip = unit[1], n = unit[2];
        int hits = 0, total;
#pragma unroll
        for (int i = 0; i < kMine; ++i) hits += id[i] == bucket;
        int at = block_scan(hits, scratch, total) - skip;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (id[i] == bucket) {
                if (at >= 0 && at < n) rows[at] = row0 + tid * kMine + i;
                ++at;
            }
        __syncthreads();
        const int cut = part * kCluster + crank, cuts = parts * kCluster;
        const int blocks = p.block[p.slices];
        const int b0 = (int)((long long)blocks * cut / cuts), b1 = (int)((long long)blocks * (cut + 1) / cuts);
        if (bucket == p.adapters) {
            const int units = p.N / 8;
            copy_rows(p, rows, n, 8 * (int)((long long)units * cut / cuts), 8 * (int)((long long)units * (cut + 1) / cuts));
        } else {
            const uint16_t *bw = p.b + bucket * p.b_adapter;
            shrink<RK>(p, p.a + bucket * p.a_adapter, rows, n, crank, h, red);
            exchange<RK>(p, p.scale ? __ldg(p.scale + bucket) : 1.f, n, h, frag, inv, crank);
            expand<RK>(p, bw, rows, n, frag, inv, b0, b1);
        }
        __syncthreads();
    }
    cluster.sync();  // (a CTA stays while others may read its share of the ids)
}

int round_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Clusters of this kernel that the device holds at once (cached per kernel, size and device).
int resident_clusters(const void *kernel, int smem) {
    struct Entry {
        const void *kernel;
        int smem, dev, n;
    };
    static std::mutex mu;
    static Entry cache[64];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].kernel == kernel && cache[i].smem == smem && cache[i].dev == dev) return cache[i].n;
    if (!set_smem_once(kernel, smem)) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster * 64, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 0;
    }
    if (used < 64) cache[used++] = Entry{kernel, smem, dev, n};
    return n;
}

}  // namespace

// Reads and clears this translation unit's record of bad indexes.
int lora_bad_index() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_bad_index, sizeof(int)) != cudaSuccess) return -1;
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_bad_index, &zero, sizeof(int));
    }
    return v;
}
}  // namespace w4a16

using namespace w4a16;

extern "C" int f16_lora(const uint16_t *x, int64_t x_row, const uint16_t *y, int64_t y_row, uint16_t *out,
                        int64_t out_row, const f16_adapters *s, const int32_t *ids, int M, void *stream) {
    if (!s) return W4_ERR_NULL;
    if (M < 0 || s->adapters < 1 || s->adapters > kMaxAdapters || s->rank < 8 || s->rank > kMaxRank ||
        s->rank % 8 != 0 || s->K < 8 || s->K % 8 != 0 || s->N < 8 || s->N % 8 != 0 || s->slices < 1 ||
        s->slices > kMaxSlices)
        return W4_ERR_SHAPE;
    LoraArgs p = {};
    for (int i = 0; i < s->slices; ++i) {
        p.col[i + 1] = s->columns[i];
        if (s->columns[i] <= p.col[i] || s->columns[i] % 8 != 0) return W4_ERR_SHAPE;
        p.block[i + 1] = p.block[i] + (p.col[i + 1] - p.col[i] + kColBlock - 1) / kColBlock;
    }
    if (p.col[s->slices] != s->N) return W4_ERR_SHAPE;
    if (M == 0) return W4A16_OK;
    if (!x || !y || !out || !ids || !s->a || !s->b) return W4_ERR_NULL;
    const auto stride_ok = [](int64_t v) { return v > 0 && v % 8 == 0; };
    if (!aligned16(x) || !aligned16(y) || !aligned16(out) || !aligned16(s->a) || !aligned16(s->b) ||
        (reinterpret_cast<uintptr_t>(ids) & 3u) != 0 || (reinterpret_cast<uintptr_t>(s->scale) & 3u) != 0 ||
        !stride_ok(x_row) || !stride_ok(y_row) || !stride_ok(out_row) || !stride_ok(s->a_adapter) ||
        !stride_ok(s->b_adapter))
        return W4_ERR_ALIGN;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    p.x = x;
    p.y = y;
    p.out = out;
    p.a = s->a;
    p.b = s->b;
    p.scale = s->scale;
    p.ids = ids;
    p.x_row = x_row;
    p.y_row = y_row;
    p.out_row = out_row;
    p.a_adapter = s->a_adapter;
    p.b_adapter = s->b_adapter;
    p.M = M;
    p.K = s->K;
    p.N = s->N;
    p.adapters = s->adapters;
    p.rank = s->rank;
    p.slices = s->slices;
    p.copy = out != y || out_row != y_row;
    const int rk = round_rank(s->rank), R = rk * s->slices;
    // 64 rows, or 32 where h and its fragments would not fit (384 ranks and more).
    p.tile = R <= 384 ? 64 : 32;
    const int passes = 16 * (rk >= 64 ? 4 : rk / 16) * 128 * 4;  // the warps' partial sums of a pass
    const int bytes_h = p.tile * R * 4;
    p.off_red = (uint32_t)bytes_h;
    p.off_hist = p.off_red + (uint32_t)(bytes_h > passes ? bytes_h : passes);
    const int smem = (int)p.off_hist + (s->adapters + 1) * 4;
    const auto kernel = rk == 16 ? lora_kernel<16> : rk == 32 ? lora_kernel<32> : rk == 64 ? lora_kernel<64>
                                                                                          : lora_kernel<128>;
    const void *fn = reinterpret_cast<const void *>(kernel);
    if (!set_smem_once(fn, smem)) return W4_ERR_LAUNCH;
    const int resident = resident_clusters(fn, smem);
    if (resident < 1) return W4_ERR_LAUNCH;
    // Parts of an item's columns: as many as give each warp one block.
    const int blocks = p.block[s->slices];
    p.parts = (blocks + kCluster * kWarps - 1) / (kCluster * kWarps);
    const int scopes = (int)((M + (long long)kScope - 1) / kScope);
    p.scope = (M + scopes - 1) / scopes;
    if (scopes == 1) {
        const long long items = min((long long)M, (long long)s->adapters + 1 + M / p.tile);  // the most there can be
        p.clusters = (int)min((long long)resident, items * p.parts);
    } else {
        p.clusters = (p.scope + p.tile - 1) / p.tile;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)scopes * p.clusters * kCluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return W4_ERR_LAUNCH;
    }
    return W4A16_OK;
}
