// f16_lora: low-rank adapters of many requests beside a shared projection,
//     out[m] = y[m] + s_a (x[m] A_a^T) B_a^T,   a = ids[m]  (negative: out = y).
// The columns may be cut into slices (q | k | v, gate | up) with an A each: B's
// rows of a slice multiply that slice's h = x A^T.
//
// What bounds it: y is read and out written once, x read once, each adapter in
// use read once; the products (2 r flops an element of x and of y) are small
// beside that up to ranks of about 64.  So the rows of one adapter are gathered,
// h stays on the chip, and one launch does everything:
//  * A cluster of up to 8 CTAs takes a unit: up to `tile` rows of one adapter, and
//    all or one of several parts of the columns.  Its CTAs split K for h (shrink),
//    add their partial sums through distributed shared memory (exchange), and split
//    the columns for the second product (expand), so nothing passes through memory
//    and no CTA waits for one outside its cluster.  Parts of one item each make h
//    themselves: A comes from L2 then, and h is far less work than the columns.
//  * Which rows belong to which adapter is found by every CTA itself, for a scope
//    of up to 1024 rows: a histogram of ids in shared memory, a prefix sum
//    over the adapters, and the rows of the unit in order by a second one (up to 32
//    rows: matches within a warp).  Any mix of ids is served.  The CTAs of a cluster
//    read a share of the ids each and take the rest from one another, so that they
//    agree on their units, and meet at the same cluster barriers, even if another
//    stream wrote ids meanwhile.
//  * Both products are mma.sync m16n8k16.  With ranks of 16 to 64 a tcgen05 tile
//    would be filled to an eighth, and the bytes are the bound, not the tensor rate.
//    The order of k inside a product is free, so lane t of a quad takes 16 contiguous
//    bytes of a row and treats them as the k indexes of two products: fragments
//    are single 16-byte loads.
//  * shrink: x and A pass through a ring of shared-memory stages by cp.async, rows
//    64 bytes longer than their data, so that the fragments' loads meet no bank twice.
//  * expand holds B's fragments of 32 columns in registers over all row tiles of the
//    unit, with ranks up to 32 the
//    next columns' on the way.  The order of columns inside the four
//    products is chosen so that a lane holds 8 neighbouring ones of two rows; its
//    16 bytes of y come ahead through a ring of its own by cp.async.
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
constexpr int kMaxCluster = 8;
constexpr int kScope = 1024;        // rows whose ids a CTA sorts
constexpr int kMaxAdapters = 4096;  // buckets of the histogram
constexpr int kMaxSlices = 4;
constexpr int kMaxRank = 128;
constexpr int kColBlock = 32;  // columns of a warp's step
constexpr int kPad = 64;       // bytes after a row of a stage
constexpr int kSmemOfTwo = 105 * 1024, kSmemOfOne = 221 * 1024;  // dynamic shared memory of two CTAs on an SM, and of one

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
    int tile;                   // rows of a unit: 64 or 32
    int parts;                  // most parts of an item's columns
    int copy;                   // out is not y: rows without an adapter are copied
    int room, pool;             // bytes of shared memory for shrink's ring; behind the fragments for expand's rings
    uint32_t off_h, off_red, off_hist;  // byte offsets in shared memory (ring and fragments at 0)
};

template <int N>
struct Int {
    static constexpr int value = N;
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
// Until at most `left` of this thread's newest groups are on the way.
__device__ __forceinline__ void copies_wait(int left) {
    switch (left) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    }
}
constexpr int kMostStages = 8;  // (copies_wait's most and two)

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

// The products of a warp with one stage of shrink: MT tiles of 16 ranks from arow
// on, NT tiles of 8 rows of x from xrow on, the 32-k blocks b = first, first + step, ...
// No branch stands between loads and products, so that they overlap; what rows past
// the last hold does not matter, as each goes into sums of its own.
template <int MT, int NT, int MAX>
__device__ __forceinline__ void stage_products(float (&acc)[MAX][4][4], uint32_t arow, uint32_t xrow, int pitch,
                                               int first, int blocks, int step) {
    for (int b = first; b < blocks; b += step) {
        uint4 x[NT], u[MT], l[MT];
#pragma unroll
        for (int i = 0; i < NT; ++i) x[i] = lds128(xrow + 8 * i * pitch + 64 * b);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            u[m] = lds128(arow + 16 * m * pitch + 64 * b);
            l[m] = lds128(arow + (16 * m + 8) * pitch + 64 * b);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i) mma_16816(acc[m][i], u[m].x, l[m].x, u[m].y, l[m].y, x[i].x, x[i].y);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i) mma_16816(acc[m][i], u[m].z, l[m].z, u[m].w, l[m].w, x[i].z, x[i].w);
    }
}

// How the 8 warps share a unit of n rows and `tiles` tiles of 16 ranks: groups of 32
// rows, groups of mt rank tiles, and groups of the 32-k blocks of a stage, whose sums
// are added at the end.  wide: the rank tiles of a group that are computed (sums of
// rank 128 come in 2, 4 and 6); held: rows of a stage, A's and then x's from xrow on.
// (Rows past the last of either are not filled, but what a warp reads ends inside.)
struct Shape {
    int rgroups, mgroups, kgroups, mt, wide, xrow, held;
};
__host__ __device__ inline Shape shape_of(int n, int tiles, int rk) {
    Shape s;
    s.rgroups = n > 32 ? 2 : 1;
    s.mgroups = tiles > 8 && n <= 32 ? 8 : tiles > 2 ? 4 : 2;
    s.kgroups = kWarps / (s.rgroups * s.mgroups);
    s.mt = (tiles + s.mgroups - 1) / s.mgroups;
    s.wide = rk < 128 ? s.mt : s.mt <= 2 ? 2 : s.mt <= 4 ? 4 : 6;
    s.xrow = 16 * tiles;
    const int a = 16 * ((tiles - 1) / s.mt * s.mt + s.wide), x = s.xrow + (n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64);
    s.held = a > x ? a : x;
    return s;
}

// Shrink: h[row][f], f = slice * rank + r, the sums over the CTA's share of K, for
// the unit's n rows.  The A of all slices are one list of slices * rank rows.
template <int RK>
__device__ __forceinline__ void shrink(const LoraArgs &p, const uint16_t *a, const int *rows, int n, int crank,
                                       int csize, uint8_t *smem) {
    constexpr int MT = RK == 16 ? 1 : RK == 32 ? 2 : RK == 64 ? 4 : 6;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int F = p.slices * p.rank, tiles = (F + 15) / 16;
    const Shape sh = shape_of(n, tiles, RK);
    const int mt = sh.mt, kgroups = sh.kgroups, xrow = sh.xrow, held = sh.held;
    const int rg = warp % sh.rgroups, mg = warp / sh.rgroups % sh.mgroups, kg = warp / (sh.rgroups * sh.mgroups);
    const int kb = (p.K + 31) / 32;
    const int k0 = 32 * (int)((long long)kb * crank / csize);
    const int k1 = min(p.K, 32 * (int)((long long)kb * (crank + 1) / csize));
    // Stages of 128 k, or of 64 where the room is short.
    const int log = p.room >= 3 * held * (256 + kPad) ? 4 : 3;  // 16-byte pieces of a row
    const int kc = 8 << log, pitch = 2 * kc + kPad, stage = held * pitch;
    const int stages = min(kMostStages, p.room / stage);  // at least 2
    const int chunks = (k1 - k0 + kc - 1) / kc;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    const int piece = threadIdx.x & ((1 << log) - 1), first = threadIdx.x >> log, step = kThreads >> log;
    auto copy_stage = [&](int c, uint32_t slot) {
        const int k = k0 + c * kc + 8 * piece;
        const bool in = k < k1;
        uint32_t dst = slot + first * pitch + 16 * piece;
        const uint16_t *src = a + (long long)first * p.K + (in ? k : 0);
        for (int r = first; r < F; r += step, dst += step * pitch, src += (long long)step * p.K) copy16(dst, src, in);
        dst = slot + (xrow + first) * pitch + 16 * piece;
        for (int r = first; r < n; r += step, dst += step * pitch) copy16(dst, p.x + rows[r] * p.x_row + (in ? k : 0), in);
    };
    uint32_t fill = base, at = base;  // the slot that is filled next, and the one that is read
    const uint32_t end = base + stages * stage;
    for (int c = 0; c < stages - 1; ++c, fill += stage) {
        if (c < chunks) copy_stage(c, fill);
        copies_commit();
    }
    float acc[MT][4][4] = {};
    const int blocks = mg * mt < tiles ? kc / 32 : 0;  // (a warp without a tile has none)
    const int arow = (16 * mg * mt + g) * pitch + 16 * t, xat = (xrow + 32 * rg + g) * pitch + 16 * t;
    auto run = [&](auto mts, auto nts) {
        constexpr int A = decltype(mts)::value, X = decltype(nts)::value;
        for (int c = 0; c < chunks; ++c) {
            copies_wait(stages - 2);
            __syncthreads();  // stage c has landed, and every warp is done with the one that is filled next
            if (c + stages - 1 < chunks) copy_stage(c + stages - 1, fill);
            copies_commit();
            fill = fill + stage == end ? base : fill + stage;
            stage_products<A, X>(acc, at + arow, at + xat, pitch, kg, blocks, kgroups);
            at = at + stage == end ? base : at + stage;
        }
    };
    auto for_rows = [&](auto mts) {
        if (n <= 8) run(mts, Int<1>());
        else if (n <= 16) run(mts, Int<2>());
        else run(mts, Int<4>());
    };
    if constexpr (MT == 1) {
        for_rows(Int<1>());
    } else if constexpr (MT == 2) {
        if (mt == 1) for_rows(Int<1>());
        else for_rows(Int<2>());
    } else if constexpr (MT == 4) {
        if (mt == 1) for_rows(Int<1>());
        else if (mt == 2) for_rows(Int<2>());
        else if (mt == 3) for_rows(Int<3>());
        else for_rows(Int<4>());
    } else {
        if (sh.wide == 2) for_rows(Int<2>());
        else if (sh.wide == 4) for_rows(Int<4>());
        else for_rows(Int<6>());
    }
    copies_wait(0);
    __syncthreads();  // the ring is free: h and the warps' sums take its place
    float *h = reinterpret_cast<float *>(smem + p.off_h);
    float *mine = kgroups == 1 ? h : reinterpret_cast<float *>(smem + p.off_red) + kg * n * F;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m >= mt) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (32 * rg + 8 * i >= n) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 32 * rg + 8 * i + 2 * t + (e & 1), f = 16 * (mg * mt + m) + g + 8 * (e >> 1);
                if (row < n && f < F) mine[row * F + f] = acc[m][i][e];
            }
        }
    }
    if (kgroups == 1) return;
    __syncthreads();
    const float *red = reinterpret_cast<const float *>(smem + p.off_red);
    for (int e = threadIdx.x; e < n * F; e += kThreads) {
        float v = 0.f;
        for (int q = 0; q < kgroups; ++q) v += red[q * n * F + e];
        h[e] = v;
    }
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

// Adds the cluster's partial sums of the rows that this CTA owns, scales and
// splits them, and leaves the fragments with every CTA of the cluster.
template <int RK>
__device__ __forceinline__ void exchange(const LoraArgs &p, float scale, int n, uint8_t *smem, float *inv, int crank,
                                         int csize) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();  // every CTA's sums are in place, and its fragments' room is free
    float *h = reinterpret_cast<float *>(smem + p.off_h);
    const int R = p.slices * RK, F = p.slices * p.rank, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = frag_pitch<RK>(p.slices);
    constexpr int J = (kMaxSlices * RK + 127) / 128;  // groups of 4 ranks of a lane
    const float inf = __int_as_float(0x7F800000);
    for (int row = crank + csize * warp; row < n; row += csize * kWarps) {
        float4 v[J];
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int r = 128 * j + 4 * lane;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R && r % RK < p.rank) {  // (ranks past the adapters' are zero)
                const float *src = h + row * F + r / RK * p.rank + r % RK;
                float4 part[kMaxCluster];
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < csize) part[c] = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(src, c));
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < csize) {
                        v[j].x += part[c].x;
                        v[j].y += part[c].y;
                        v[j].z += part[c].z;
                        v[j].w += part[c].w;
                    }
                v[j].x *= scale;
                v[j].y *= scale;
                v[j].z *= scale;
                v[j].w *= scale;
            }
            const float m = fmaxf(fmaxf(fabsf(v[j].x), fabsf(v[j].y)), fmaxf(fabsf(v[j].z), fabsf(v[j].w)));
            const bool nan = v[j].x != v[j].x || v[j].y != v[j].y || v[j].z != v[j].z || v[j].w != v[j].w;
            top = fmaxf(top, nan ? inf : m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // 2^(12 - e) for a largest value in [2^e, 2^(e + 1)); 1 for rows of zeros and those that are not finite.
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const int shift = e == 128 || top == 0.f ? 0 : 12 - max(e, -100);
        const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
        if (lane < csize) cluster.map_shared_rank(inv, lane)[row] = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int r = 128 * j + 4 * lane;
            if (r >= R) continue;
            const float a = v[j].x * up, b = v[j].y * up, c = v[j].z * up, d = v[j].w * up;
            const uint32_t h0 = pack(a, b), h1 = pack(c, d);
            const float2 f0 = unpack(h0), f1 = unpack(h1);
            const auto rest = [](float x, float hi) { return fabsf(x - hi) < 1e30f ? x - hi : 0.f; };  // (none of infinities)
            const uint4 w = make_uint4(h0, h1, pack(rest(a, f0.x), rest(b, f0.y)), pack(rest(c, f1.x), rest(d, f1.y)));
            uint8_t *dst = smem + row * pitch + frag_at<RK>(r / RK, r % RK);
#pragma unroll
            for (int q = 0; q < kMaxCluster; ++q)
                if (q < csize) *reinterpret_cast<uint4 *>(cluster.map_shared_rank(dst, q)) = w;
        }
    }
    cluster.sync();
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

// Expand: out = y + h B^T over the CTA's column blocks [b0, b1) of the unit's rows,
// whose addresses in y and out are yrow and orow.
template <int RK>
__device__ __forceinline__ void expand(const LoraArgs &p, const uint16_t *bw, const uint16_t *const *yrow,
                                       uint16_t *const *orow, int n, uint8_t *smem, const float *inv, int b0, int b1) {
    constexpr int KS = RK / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (b0 + warp >= b1) return;
    const int tiles = (n + 15) / 16, pitch = frag_pitch<RK>(p.slices);
    const uint32_t frag = (uint32_t)__cvta_generic_to_shared(smem) + g * pitch + 16 * t;
    // The warp's ring of y: `depth` column blocks of up to 64 rows, 16 bytes a lane each.
    const int slot = tiles * 1024, depth = min(4, p.pool / (kWarps * slot));
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + p.off_h) + warp * depth * slot + lane * 16;
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
    load_b(own);
    for (int d = 0; d < depth; ++d) copy_y(ring + d * slot);
    uint32_t at = ring;
    while (true) {
        copies_wait(depth - 1);  // (a lane reads only what it copied itself)
        const uint32_t f0 = frag + own.slice * (64 * KS);
        const int col = own.col + 8 * t;
        const bool cv = col < own.end;
        // Two row tiles at a time; past the last one only the stores are left out.
        for (int tile = 0; tile < tiles; tile += 2) {
            float acc[2][4][4] = {};
            uint4 old[2][2];
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 2; ++i) old[w][i] = lds128(at + (2 * min(tile + w, tiles - 1) + i) * 512);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint4 u[2], l[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t row = f0 + 16 * min(tile + w, tiles - 1) * pitch + 64 * k;
                    u[w] = lds128(row);
                    l[w] = lds128(row + 8 * pitch);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_16816(acc[w][j], u[w].x, l[w].x, u[w].y, l[w].y, bf[j][k][0], bf[j][k][1]);
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_16816(acc[w][j], u[w].z, l[w].z, u[w].w, l[w].w, bf[j][k][0], bf[j][k][1]);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 16 * (tile + w) + 8 * i + g, rs = r & 63;
                    const float2 f = make_float2(inv[rs], inv[rs]);
                    const uint32_t v[4] = {old[w][i].x, old[w][i].y, old[w][i].z, old[w][i].w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 z = fma2(make_float2(acc[w][j][2 * i], acc[w][j][2 * i + 1]), f, unpack(v[j]));
                        o[j] = pack(z.x, z.y);
                    }
                    uint16_t *dst = orow[rs] + col;
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
__global__ void __launch_bounds__(kThreads, RK == 128 ? 1 : 2) lora_kernel(const __grid_constant__ LoraArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int scratch[kWarps], rows[64], unit[3];
    __shared__ float inv[64];
    __shared__ const uint16_t *yrow[64];
    __shared__ uint16_t *orow[64];
    __shared__ __align__(16) int own[kScope];  // buckets of this CTA's share of the rows, -1 past the scope
    cg::cluster_group cluster = cg::this_cluster();
    int *hist = reinterpret_cast<int *>(smem + p.off_hist);  // rows of each adapter; of none at the end
    const int tid = threadIdx.x, lane = tid & 31;
    const int csize = (int)cluster.num_blocks(), crank = (int)cluster.block_rank(), cl = (int)blockIdx.x / csize;
    const int scope = cl / p.clusters, q = cl % p.clusters;
    const int row0 = scope * p.scope, nrow = min(p.scope, p.M - row0);
    const int buckets = p.adapters + 1;
    const bool few = nrow <= 32;
    if (!few)
        for (int i = tid; i < buckets; i += kThreads) hist[i] = 0;
    pdl_wait();
    const int share = few ? 32 : kScope / csize;  // (of few rows, the first CTA's count)
    for (int i = tid; i < share; i += kThreads) {
        const int r = crank * share + i;
        int bucket = -1;
        if (r < nrow) {
            const int v = __ldg(p.ids + row0 + r);
            if (v >= p.adapters) atomicExch(&g_bad_index, 1);
            bucket = v < 0 || v >= p.adapters ? p.adapters : v;
        }
        own[i] = bucket;
    }
    cluster.sync();
    constexpr int kMine = kScope / kThreads;
    static_assert(kMine == 4, "a thread's rows come from one CTA in one read");
    int id[kMine], mine = 0, first = 0, items;
    unsigned leaders = 0, same = 0;
    const int per = (buckets + kThreads - 1) / kThreads;
    if (few) {
        // Every warp knows all rows: an item to each bucket, in the order of their first rows.
        id[0] = cluster.map_shared_rank(own, 0)[lane];
        same = __match_any_sync(~0u, id[0]);
        leaders = __ballot_sync(~0u, id[0] >= 0 && (id[0] < p.adapters || p.copy) && (same & ((1u << lane) - 1u)) == 0u);
        items = __popc(leaders);
    } else {
        // Four rows a thread, in order.
        const int4 four = *reinterpret_cast<const int4 *>(cluster.map_shared_rank(own, tid * kMine / share) +
                                                          tid * kMine % share);
        id[0] = four.x, id[1] = four.y, id[2] = four.z, id[3] = four.w;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            if (id[i] >= 0) atomicAdd(hist + id[i], 1);
        __syncthreads();
        // Items: up to `tile` rows of one bucket.  This thread's buckets are in a row.
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < buckets && (b < p.adapters || p.copy)) mine += (hist[b] + p.tile - 1) / p.tile;
        }
        first = block_scan(mine, scratch, items);
    }
    const int parts = max(1, min(p.parts, p.clusters / max(items, 1)));
    for (int u = q; u < items * parts; u += p.clusters) {
        const int item = u % items, part = u / items;
        int bucket, n;
        if (few) {
            unsigned left = leaders;
            for (int i = 0; i < item; ++i) left &= left - 1u;
            const int lead = __ffs(left) - 1;
            bucket = __shfl_sync(~0u, id[0], lead);
            const unsigned its = __shfl_sync(~0u, same, lead);
            n = __popc(its);
            if (tid < 32 && its >> lane & 1u) rows[__popc(its & ((1u << lane) - 1u))] = row0 + lane;
            __syncthreads();
        } else {
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
            bucket = unit[0], n = unit[2];
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
        }
        const int cut = part * csize + crank, cuts = parts * csize;
        if (bucket == p.adapters) {
            const int units = p.N / 8;
            copy_rows(p, rows, n, 8 * (int)((long long)units * cut / cuts), 8 * (int)((long long)units * (cut + 1) / cuts));
        } else {
            const int blocks = p.block[p.slices];
            if (tid < n) {  // (read after the barriers of shrink)
                yrow[tid] = p.y + rows[tid] * p.y_row;
                orow[tid] = p.out + rows[tid] * p.out_row;
            }
            shrink<RK>(p, p.a + bucket * p.a_adapter, rows, n, crank, csize, smem);
            exchange<RK>(p, p.scale ? __ldg(p.scale + bucket) : 1.f, n, smem, inv, crank, csize);
            expand<RK>(p, p.b + bucket * p.b_adapter, yrow, orow, n, smem, inv, (int)((long long)blocks * cut / cuts),
                       (int)((long long)blocks * (cut + 1) / cuts));
        }
        __syncthreads();
    }
    cluster.sync();  // (a CTA stays while others may read its share of the ids)
}

int round_rank(int rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }

// Clusters of this kernel that the device holds at once (cached per kernel, size and device).
int resident_clusters(const void *kernel, int smem, int cluster) {
    struct Entry {
        const void *kernel;
        int smem, cluster, dev, n;
    };
    static std::mutex mu;
    static Entry cache[64];
    static int used = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].kernel == kernel && cache[i].smem == smem && cache[i].cluster == cluster && cache[i].dev == dev)
            return cache[i].n;
    if (!set_smem_once(kernel, smem)) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster * 64, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return 0;
    }
    if (used < 64) cache[used++] = Entry{kernel, smem, cluster, dev, n};
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
    const int rk = round_rank(s->rank), R = rk * s->slices, F = s->rank * s->slices;
    // 64 rows, or 32 where h and its fragments would not fit (more than 384 ranks).
    p.tile = R <= 384 ? 64 : 32;
    const int pitch = rk == 16   ? frag_pitch<16>(s->slices)
                      : rk == 32 ? frag_pitch<32>(s->slices)
                      : rk == 64 ? frag_pitch<64>(s->slices)
                                 : frag_pitch<128>(s->slices);
    const int frag = p.tile * pitch, h = p.tile * F * 4, hist = (s->adapters + 1) * 4;
    p.off_h = (uint32_t)frag;
    p.off_red = (uint32_t)(frag + h);
    // The ring of x and A (at least two stages of 64 k), then h with the warps' sums,
    // then expand's rings (at least a block a warp) lie in the same place behind the
    // fragments, or over them.  Two CTAs on an SM if that is enough, else one; rank
    // 128 has one, for its registers.
    const int tiles = (F + 15) / 16;
    const int held = max(shape_of(32, tiles, rk).held, shape_of(p.tile, tiles, rk).held);
    const int red = (F <= 32 ? 128 : F <= 128 ? 64 : 0) * F * 4;  // [k groups][rows][ranks]
    const int need = max(2 * held * (128 + kPad), max(frag + h + red, frag + kWarps * p.tile * 64));
    p.room = (rk < 128 && need + hist <= kSmemOfTwo ? kSmemOfTwo : kSmemOfOne) - hist;
    p.pool = p.room - frag;
    p.off_hist = (uint32_t)p.room;
    const int smem = p.room + hist;
    const auto kernel = rk == 16 ? lora_kernel<16> : rk == 32 ? lora_kernel<32> : rk == 64 ? lora_kernel<64>
                                                                                          : lora_kernel<128>;
    const void *fn = reinterpret_cast<const void *>(kernel);
    if (!set_smem_once(fn, smem)) return W4_ERR_LAUNCH;
    // Clusters of 8, or of fewer CTAs where as many row tiles fill the GPU.
    const int scopes = (int)((M + (long long)kScope - 1) / kScope);
    p.scope = (M + scopes - 1) / scopes;
    const int most = (p.scope + p.tile - 1) / p.tile;  // items of a scope whose rows are of one adapter
    int cluster = kMaxCluster, resident = 0;
    for (;; cluster /= 2) {
        resident = resident_clusters(fn, smem, cluster);
        if (resident < 1) return W4_ERR_LAUNCH;
        if (cluster == 1 || (long long)scopes * most <= resident) break;
    }
    // Parts of an item's columns: as many as give each warp one block.
    p.parts = (p.block[s->slices] + cluster * kWarps - 1) / (cluster * kWarps);
    if (scopes == 1) {
        const long long items = min((long long)M, (long long)s->adapters + 1 + M / p.tile);  // the most there can be
        p.clusters = (int)min((long long)resident, items * p.parts);
    } else {
        p.clusters = most;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)scopes * p.clusters * cluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
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
