// f16_rope, f16_kv_append: rotary positions, and new tokens' keys and values
// written into the paged cache with the rotation applied on the way.
//
// The angle of pair i at position p is p * theta_i.  Held as a fraction of a
// turn in 64 bits, F_i = round(2^64 theta_i / 2 pi), its reduction to one
// turn is the wrap of an integer product, p * F_i mod 2^64, which adds no error
// at any p: the angle is off by |p| times the error of F_i, half a unit of
// 2^-64 turns in a correctly rounded table, up to some 2^9 units in one made
// in binary64 (2^-24 turns at the largest p).  The product's upper half, as a
// signed fraction of half a turn, goes to sincospif.
//
// Both calls move every element once in and once out and are bound by that.
// A lane owns one unit of a head: 8 elements, 16 bytes, which are 4 rotated
// pairs (of adjacent elements, or 4 elements of each half) or 8 elements to
// copy.  A warp takes one token and up to HPL * (256 / head_dim) of its heads,
// so a lane turns the same pairs of each of its heads and computes
// their sines once; all its loads are issued before the sines and the index
// look-ups that do not depend on them.
//
// Measured: rope of 16384 tokens x 16 heads of 128, 134 MB, 21.6 us, 6.2 TB/s;
// append of 16384 tokens, 16 + 2 x 8 heads, 268 MB, 43.7 us, 6.1 TB/s, against
// 6.69 TB/s of a plain copy.  Steps of a few tokens: 1.5 and 2.5 us in a graph,
// the launch and one chain of dependent reads.
#include <string.h>

#include "kv.cuh"

namespace w4a16 {
namespace {

// Heads of a lane (HPL below): the most whose warps fill half the GPU.  More
// heads: the look-ups and sines of a warp serve more of its bytes (append,
// 16384 tokens of 16 + 2 x 8 heads of 128: 43.7 us with 8, 53.6 with 4, 78.6
// with 2, 79 with 16 (fewer loads fit the registers); 2000 tokens: 6.8 with 8,
// 8.1 with 4).  Fewer: more warps, and a shorter path from load to store
// (append in a graph, 16 tokens: 2.5 us with 1, 3.0 with 4; 1000 tokens: 4.8
// with 4, 8.8 with 1).
constexpr int kManyHeads = 8, kSomeHeads = 4;
constexpr int kWarps = 4;
constexpr int kBlocks = 8;  // resident on an SM

struct Rot {
    const uint64_t *turns;
    int rot, interleaved;
    float factor;
};

// A strided tensor [tokens][heads][head_dim].
struct Heads {
    const uint16_t *x;
    long long token, head;
};

struct Unit {
    uint2 a, b;  // half layout: 4 elements of each half; else 8 elements in order
};

// Element offsets of the two 4-element parts of unit u.
__device__ __forceinline__ int2 unit_parts(int u, const Rot &r) {
    return 8 * u < r.rot && !r.interleaved ? make_int2(4 * u, r.rot / 2 + 4 * u) : make_int2(8 * u, 8 * u + 4);
}

__device__ __forceinline__ Unit load_unit(const uint16_t *head, int2 at) {
    Unit u;
    if (at.y == at.x + 4) {  // 8 elements in order: one 16-byte access
        const uint4 v = *reinterpret_cast<const uint4 *>(head + at.x);
        u.a = make_uint2(v.x, v.y);
        u.b = make_uint2(v.z, v.w);
        return u;
    }
    u.a = *reinterpret_cast<const uint2 *>(head + at.x);
    u.b = *reinterpret_cast<const uint2 *>(head + at.y);
    return u;
}

__device__ __forceinline__ void store_unit(uint16_t *head, int2 at, const Unit &u) {
    if (at.y == at.x + 4) {
        *reinterpret_cast<uint4 *>(head + at.x) = make_uint4(u.a.x, u.a.y, u.b.x, u.b.y);
    } else {
        *reinterpret_cast<uint2 *>(head + at.x) = u.a;
        *reinterpret_cast<uint2 *>(head + at.y) = u.b;
    }
}

struct Turn {
    float c[4], s[4];
};

// Cosines and sines, times the factor, of pairs 4u .. 4u + 3 at position p.
__device__ __forceinline__ Turn turn_of(const Rot &r, int u, int p) {
    Turn t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t f = (uint64_t)(int64_t)p * __ldg(r.turns + 4 * u + i);
        const float half_turns = (float)(int32_t)(f >> 32) * 0x1p-31f;
        sincospif(half_turns, &t.s[i], &t.c[i]);
        t.c[i] *= r.factor;
        t.s[i] *= r.factor;
    }
    return t;
}

__device__ __forceinline__ float2 f2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The rotated unit: fp32 products and sums, one rounding to binary16.
__device__ __forceinline__ Unit turned(const Unit &u, const Turn &t, int interleaved) {
    Unit o;
    const float2 v0 = f2(u.a.x), v1 = f2(u.a.y), v2 = f2(u.b.x), v3 = f2(u.b.y);
    if (interleaved) {
        o.a.x = h2(v0.x * t.c[0] - v0.y * t.s[0], v0.x * t.s[0] + v0.y * t.c[0]);
        o.a.y = h2(v1.x * t.c[1] - v1.y * t.s[1], v1.x * t.s[1] + v1.y * t.c[1]);
        o.b.x = h2(v2.x * t.c[2] - v2.y * t.s[2], v2.x * t.s[2] + v2.y * t.c[2]);
        o.b.y = h2(v3.x * t.c[3] - v3.y * t.s[3], v3.x * t.s[3] + v3.y * t.c[3]);
    } else {  // pairs (v0.x, v2.x), (v0.y, v2.y), (v1.x, v3.x), (v1.y, v3.y)
        o.a.x = h2(v0.x * t.c[0] - v2.x * t.s[0], v0.y * t.c[1] - v2.y * t.s[1]);
        o.a.y = h2(v1.x * t.c[2] - v3.x * t.s[2], v1.y * t.c[3] - v3.y * t.s[3]);
        o.b.x = h2(v0.x * t.s[0] + v2.x * t.c[0], v0.y * t.s[1] + v2.y * t.c[1]);
        o.b.y = h2(v1.x * t.s[2] + v3.x * t.c[2], v1.y * t.s[3] + v3.y * t.c[3]);
    }
    return o;
}

// Warp w of the grid takes heads [g * per, (g + 1) * per) of token w / groups,
// g = w % groups; lane l the unit l % units of every (32 / units)-th of them.
template <int HPL>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
    rope_kernel(Heads x, Heads y, const int32_t *__restrict__ positions, Rot r, int tokens, int heads, int units,
                int groups) {
    pdl_wait();
    const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long t = w / (unsigned)groups;
    const int side = 32 / units, sub = lane / units, u = lane % units;
    if (t >= tokens || sub >= side) return;
    const int h0 = (int)(w % (unsigned)groups) * side * HPL + sub;
    const int2 at = unit_parts(u, r);
    Unit v[HPL];
#pragma unroll
    for (int j = 0; j < HPL; ++j)
        if (h0 + j * side < heads) v[j] = load_unit(x.x + t * x.token + (h0 + j * side) * x.head, at);
    uint16_t *dst = const_cast<uint16_t *>(y.x) + t * y.token;
    const bool rotated = 8 * u < r.rot;
    Turn turn;
    if (rotated) turn = turn_of(r, u, positions ? __ldg(positions + t) : (int)t);
#pragma unroll
    for (int j = 0; j < HPL; ++j)
        if (h0 + j * side < heads)
            store_unit(dst + (h0 + j * side) * y.head, at, rotated ? turned(v[j], turn, r.interleaved) : v[j]);
}

// The largest i with q_offsets[i] <= t, by a search whose steps the warp's
// lanes take together (32-fold: one dependent load up to 32 offsets, two up
// to 1024); -1 if there is none.
__device__ __forceinline__ int find_seq(const int32_t *q_offsets, int n, int t, int lane) {
    int lo = 0, size = n;
    while (size > 32) {
        const int step = (size + 31) / 32;
        const int i = lane * step;
        const unsigned m = __ballot_sync(~0u, i < size && __ldg(q_offsets + lo + i) <= t);
        if (m == 0) return -1;
        const int k = __popc(m) - 1;
        lo += k * step;
        size = min(step, size - k * step);
    }
    const unsigned m = __ballot_sync(~0u, lane < size && __ldg(q_offsets + lo + lane) <= t);
    return lo + __popc(m) - 1;
}

struct AppendArgs {
    Heads q, k, v;
    uint16_t *y, *kc, *vc;
    long long y_token, y_head, kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
    const int32_t *positions;
    KvBatch b;
    Rot r;  // rot 0: no rotation
    int num_pages, page_size, q_heads, kv_heads, units, groups;
};

// As rope_kernel, over the heads of q, then k, then v of one token; the
// token's sequence, and the page of its position, are found by the warp.
template <int HPL>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_wait();
    const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int t = (int)(w / (unsigned)a.groups);
    if (t >= a.b.total_q) return;
    const int side = 32 / a.units, sub = lane / a.units, u = lane % a.units;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int h0 = (int)(w % (unsigned)a.groups) * side * HPL + sub;
    const int2 at = unit_parts(u, a.r);
    Unit v[HPL];
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        const int h = h0 + j * side;
        if (sub < side && h < heads) {
            const int hk = h - a.q_heads, hv = hk - a.kv_heads;
            const uint16_t *src = hk < 0 ? a.q.x + t * a.q.token + h * a.q.head
                                  : hv < 0 ? a.k.x + t * a.k.token + hk * a.k.head
                                           : a.v.x + t * a.v.token + hv * a.v.head;
            v[j] = load_unit(src, at);
        }
    }
    const int b = find_seq(a.b.q_offsets, a.b.batch + 1, t, lane);
    if (b < 0 || b >= a.b.batch) return;  // a row outside every sequence
    const Seq s = load_seq(a.b, b);
    if (t < s.q0 || t >= s.q0 + s.qn) return;  // offsets out of order: reported by load_seq
    const int p = s.kv - s.qn + (t - s.q0);
    int page = -1;
    // (A position from a clamped length or offset may be another token's: nothing is written there.)
    if (p >= 0 && s.ordered && s.fits) {
        page = __ldg(a.b.table + (long long)b * a.b.table_stride + p / a.page_size);
        if ((unsigned)page >= (unsigned)a.num_pages) {
            page = -1;
            atomicExch(&g_bad_index, 1);
        }
    }
    if (sub >= side) return;
    const int slot = p - p / a.page_size * a.page_size;
    const bool rotated = 8 * u < a.r.rot;
    Turn turn;
    if (rotated) turn = turn_of(a.r, u, a.positions ? __ldg(a.positions + t) : p);
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        const int h = h0 + j * side;
        if (h >= heads) break;
        const int hk = h - a.q_heads, hv = hk - a.kv_heads;
        if (hk >= 0 && page < 0) break;
        uint16_t *dst = hk < 0 ? a.y + t * a.y_token + h * a.y_head
                        : hv < 0 ? a.kc + page * a.kc_page + slot * a.kc_token + hk * a.kc_head
                                 : a.vc + page * a.vc_page + slot * a.vc_token + hv * a.vc_head;
        store_unit(dst, at, rotated && hv < 0 ? turned(v[j], turn, a.r.interleaved) : v[j]);
    }
}

int check_rotation(const f16_rotation *r, int head_dim, Rot &out) {
    if (!r->turns) return W4_ERR_NULL;
    if (r->rot < 8 || r->rot > head_dim || r->rot % 8 != 0 || (r->interleaved & ~1) != 0) return W4_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0) return W4_ERR_ALIGN;
    out.turns = r->turns;
    out.rot = r->rot;
    out.interleaved = r->interleaved;
    out.factor = r->factor;
    return W4A16_OK;
}

// Warps per token for `heads` heads of `units` 16-byte units, hpl to a lane.
int head_groups(int heads, int units, int hpl) {
    const int per = 32 / units * hpl;
    return (heads + per - 1) / per;
}
// Heads of a lane of a call (see kManyHeads).
int heads_per_lane(long long tokens, int heads, int units) {
    const long long slots = (long long)sm_count() * kBlocks * kWarps;  // warps that the GPU holds
    if (tokens * head_groups(heads, units, kManyHeads) > slots / 2) return kManyHeads;
    return tokens * head_groups(heads, units, 1) > slots / 2 ? kSomeHeads : 1;
}

// Launch as a programmatic dependent (the kernels wait for the one before
// first: it only takes the launch itself off the path).
template <class K, class... A>
int launch(K kernel, long long warps, void *stream, A... args) {
    if (warps > 0x7FFFFFFFll) return W4_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + kWarps - 1) / kWarps), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
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

// Encodes a binary16 tensor map with 128-byte swizzle; false for a stride it
// cannot take (2^40 bytes and more).
bool f16_map(uint64_t (&out)[16], void *x, int rank, const uint64_t *dims, const uint64_t *strides,
             const uint32_t *box) {
    static_assert(sizeof(CUtensorMap) == sizeof(out), "tensor map size");
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    cuuint64_t d[5], s[4];
    cuuint32_t b[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i > 0) s[i - 1] = strides[i - 1];
    }
    alignas(64) CUtensorMap m;
    if (encode_fn()(&m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank, x, d, s, b, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
    memcpy(out, &m, sizeof(m));
    return true;
}

}  // namespace

// Reads and clears this translation unit's record of bad indexes.
int rope_bad_index() {
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

extern "C" int f16_rope(const uint16_t *x, int64_t x_token, int64_t x_head, uint16_t *y, int64_t y_token,
                        int64_t y_head, const int32_t *positions, const f16_rotation *rotation, int tokens, int heads,
                        int head_dim, void *stream) {
    if (!rotation) return W4_ERR_NULL;
    if (tokens < 0 || heads < 1 || heads > kMaxHeads || !head_dim_ok(head_dim)) return W4_ERR_SHAPE;
    Rot r;
    const int st = check_rotation(rotation, head_dim, r);
    if (st != W4A16_OK) return st;
    if (tokens == 0) return W4A16_OK;
    if (!x || !y) return W4_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !stride_ok(x_token) || !stride_ok(x_head) || !stride_ok(y_token) ||
        !stride_ok(y_head) || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
        return W4_ERR_ALIGN;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    const int units = head_dim / 8, hpl = heads_per_lane(tokens, heads, units), groups = head_groups(heads, units, hpl);
    return launch(hpl == kManyHeads   ? rope_kernel<kManyHeads>
                  : hpl == kSomeHeads ? rope_kernel<kSomeHeads>
                                      : rope_kernel<1>,
                  (long long)tokens * groups, stream, Heads{x, x_token, x_head}, Heads{y, y_token, y_head}, positions, r,
                  tokens, heads, units, groups);
}

extern "C" int f16_kv_append(const uint16_t *k, int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token,
                             int64_t v_head, const f16_kv_cache *cache, const f16_kv_batch *batch,
                             const f16_rotation *rotation, const int32_t *positions, const uint16_t *q,
                             int64_t q_token, int64_t q_head, uint16_t *y, int64_t y_token, int64_t y_head,
                             int q_heads, void *stream) {
    int st = check_cache(cache);
    if (st != W4A16_OK) return st;
    AppendArgs a;
    st = check_batch(batch, cache->page_size, a.b);
    if (st != W4A16_OK) return st;
    a.r = Rot{nullptr, 0, 0, 1.f};
    if (rotation && (st = check_rotation(rotation, cache->head_dim, a.r)) != W4A16_OK) return st;
    if (q && (q_heads < 1 || q_heads > kMaxHeads)) return W4_ERR_SHAPE;
    if (batch->total_q == 0) return W4A16_OK;
    if (!k || !v || (q && !y)) return W4_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(y) || !stride_ok(k_token) ||
        !stride_ok(k_head) || !stride_ok(v_token) || !stride_ok(v_head) ||
        (q && (!stride_ok(q_token) || !stride_ok(q_head) || !stride_ok(y_token) || !stride_ok(y_head))) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
        return W4_ERR_ALIGN;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    a.q = Heads{q, q_token, q_head};
    a.k = Heads{k, k_token, k_head};
    a.v = Heads{v, v_token, v_head};
    a.y = y;
    a.y_token = y_token;
    a.y_head = y_head;
    a.kc = cache->k;
    a.vc = cache->v;
    a.kc_page = cache->k_page;
    a.kc_token = cache->k_token;
    a.kc_head = cache->k_head;
    a.vc_page = cache->v_page;
    a.vc_token = cache->v_token;
    a.vc_head = cache->v_head;
    a.positions = positions;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.q_heads = q ? q_heads : 0;
    a.kv_heads = cache->heads;
    a.units = cache->head_dim / 8;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int hpl = heads_per_lane(batch->total_q, heads, a.units);
    a.groups = head_groups(heads, a.units, hpl);
    return launch(hpl == kManyHeads   ? append_kernel<kManyHeads>
                  : hpl == kSomeHeads ? append_kernel<kSomeHeads>
                                      : append_kernel<1>,
                  (long long)batch->total_q * a.groups, stream, a);
}

extern "C" int f16_kv_cache_init(f16_kv_cache *c, uint16_t *k, uint16_t *v, const int64_t ks[3], const int64_t vs[3],
                                 int num_pages, int page_size, int heads, int head_dim) {
    if (!c || !k || !v || !ks || !vs) return W4_ERR_NULL;
    if (num_pages < 1 || page_size < 8 || page_size % 8 != 0 || heads < 1 || heads > kMaxHeads ||
        !head_dim_ok(head_dim))
        return W4_ERR_SHAPE;
    if (!aligned16(k) || !aligned16(v)) return W4_ERR_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (!stride_ok(ks[i]) || !stride_ok(vs[i])) return W4_ERR_ALIGN;
    if (!encode_fn()) return W4_ERR_DEVICE;
    c->k = k;
    c->v = v;
    c->k_page = ks[0];
    c->k_token = ks[1];
    c->k_head = ks[2];
    c->v_page = vs[0];
    c->v_token = vs[1];
    c->v_head = vs[2];
    c->num_pages = num_pages;
    c->page_size = page_size;
    c->heads = heads;
    c->head_dim = head_dim;
    c->box_rows = kv_box_rows(page_size, head_dim);
    c->reserved = 0;
    // Copies of box_rows tokens of one head of one page, 128-byte swizzle: 64
    // elements of each (elements past head_dim read as zero: heads are padded
    // to 64), or all head_dim elements as columns of 64, one after the other.
    for (int i = 0; i < 2; ++i) {
        const int64_t *s = i ? vs : ks;
        uint16_t *x = i ? v : k;
        const uint64_t st[5] = {2, (uint64_t)s[1] * 2, 128, (uint64_t)s[2] * 2, (uint64_t)s[0] * 2};
        const uint64_t dims[4] = {(uint64_t)head_dim, (uint64_t)page_size, (uint64_t)heads, (uint64_t)num_pages};
        const uint64_t strides[3] = {st[1], st[3], st[4]};
        const uint32_t box[4] = {64, (uint32_t)c->box_rows, 1, 1};
        if (!f16_map(i ? c->v_map : c->k_map, x, 4, dims, strides, box)) return W4_ERR_SHAPE;
        if (head_dim % 64 != 0 || head_dim == 64) continue;
        const uint64_t wide_dims[5] = {64, (uint64_t)page_size, (uint64_t)head_dim / 64, (uint64_t)heads,
                                       (uint64_t)num_pages};
        const uint32_t wide_box[5] = {64, (uint32_t)c->box_rows, (uint32_t)head_dim / 64, 1, 1};
        if (!f16_map(i ? c->v_wide : c->k_wide, x, 5, wide_dims, st + 1, wide_box)) return W4_ERR_SHAPE;
    }
    return W4A16_OK;
}
