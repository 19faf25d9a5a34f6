// f16_rope, f16_kv_append: rotary positions, and new tokens' keys and values
// written into the paged cache with the rotation applied on the way; in the
// _ex calls every query and key head is normed before it is turned.
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
// The norm of a head, z = x w / sqrt(mean x^2 + eps), needs one sum over the
// head's lanes, which hold it whole: each lane sums its 8 squares, and shuffles
// inside the warp add the lanes (4 of them a head of 128), so the norm costs no
// memory but its weights, which stay in L1.  Squares, sum, root and products are
// fp32, and the normed and turned value is rounded once, to binary16.
//
// Measured: rope of 16384 tokens x 16 heads of 128, 134 MB, 21.5 us, 6.2 TB/s;
// append of 16384 tokens, 16 + 2 x 8 heads, 268 MB, 43.7 us, 6.1 TB/s, against
// 6.69 TB/s of a plain copy.  Steps of a few tokens: 1.7 and 2.4 us in a graph,
// the launch and one chain of dependent reads.  With norms: the same rope 25.2 us;
// an append of 14 + 2 x 2 heads of 64, 25000 tokens, 37.0 us (25.3 without): instructions.
#include <math.h>
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
constexpr int kAppendBlocks = 7;  // (append of 25000 tokens, 14 + 2 x 2 heads of 64: 25.2 us; 8: 26.9, spilling; 6: 26.7)
constexpr int kNormBlocks = 6;  // with norms, whose sums and weights take registers (the same append: 36.9; 8: 39.6; 5: 38.1)

struct Rot {
    const uint64_t *turns;  // rot 0: no rotation
    int rot, interleaved;
    float factor;
};

struct Norm {
    const float *w;  // [head_dim]; null: no norm
    float eps;
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

// Cosine (x) and sine (y), times the factor, of pair i at position p.
__device__ __forceinline__ float2 turn_of(const Rot &r, int i, int p) {
    const uint64_t f = (uint64_t)(int64_t)p * __ldg(r.turns + i);
    const float half_turns = (float)(int32_t)(f >> 32) * 0x1p-31f;
    float2 t;
    sincospif(half_turns, &t.y, &t.x);
    return make_float2(t.x * r.factor, t.y * r.factor);
}

// Those of the lane's unit, pairs 4u .. 4u + 3.  The lanes that hold the same
// unit of different heads (sub = 0 .. side - 1) turn alike, and four or two of
// them share the sines out among themselves (SHARE: not where a lane has one head
// and the path from its load to its store counts: 2.41 us against 2.76 for a
// step of 16 tokens).  Every lane of the warp takes part.
template <bool SHARE>
__device__ __forceinline__ Turn turns_of(const Rot &r, int u, int units, int side, int sub, bool rotated, int p) {
    Turn t;
    float2 v = make_float2(1.f, 0.f);
    if (SHARE && side >= 4) {
        if (rotated) v = turn_of(r, 4 * u + (sub & 3), p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[i] = __shfl_sync(~0u, v.x, i * units + u);
            t.s[i] = __shfl_sync(~0u, v.y, i * units + u);
        }
    } else if (SHARE && side >= 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (rotated) v = turn_of(r, 4 * u + 2 * (sub & 1) + k, p);
            t.c[k] = __shfl_sync(~0u, v.x, u);
            t.s[k] = __shfl_sync(~0u, v.y, u);
            t.c[2 + k] = __shfl_sync(~0u, v.x, units + u);
            t.s[2 + k] = __shfl_sync(~0u, v.y, units + u);
        }
    } else if (rotated) {  // (one branch, so that the four loads go out together)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v = turn_of(r, 4 * u + i, p);
            t.c[i] = v.x;
            t.s[i] = v.y;
        }
    }
    return t;
}

__device__ __forceinline__ float2 f2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ uint32_t h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The 8 elements of a unit: v[0..3] of part a, v[4..7] of part b.
struct Vals {
    float v[8];
};
__device__ __forceinline__ Vals vals(const Unit &u) {
    const float2 v0 = f2(u.a.x), v1 = f2(u.a.y), v2 = f2(u.b.x), v3 = f2(u.b.y);
    return Vals{{v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y}};
}

// The rotated unit: fp32 products and sums, one rounding to binary16.
__device__ __forceinline__ Unit turned(const Vals &x, const Turn &t, int interleaved) {
    const float *v = x.v;
    Unit o;
    if (interleaved) {
        o.a.x = h2(v[0] * t.c[0] - v[1] * t.s[0], v[0] * t.s[0] + v[1] * t.c[0]);
        o.a.y = h2(v[2] * t.c[1] - v[3] * t.s[1], v[2] * t.s[1] + v[3] * t.c[1]);
        o.b.x = h2(v[4] * t.c[2] - v[5] * t.s[2], v[4] * t.s[2] + v[5] * t.c[2]);
        o.b.y = h2(v[6] * t.c[3] - v[7] * t.s[3], v[6] * t.s[3] + v[7] * t.c[3]);
    } else {  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
        o.a.x = h2(v[0] * t.c[0] - v[4] * t.s[0], v[1] * t.c[1] - v[5] * t.s[1]);
        o.a.y = h2(v[2] * t.c[2] - v[6] * t.s[2], v[3] * t.c[3] - v[7] * t.s[3]);
        o.b.x = h2(v[0] * t.s[0] + v[4] * t.c[0], v[1] * t.s[1] + v[5] * t.c[1]);
        o.b.y = h2(v[2] * t.s[2] + v[6] * t.c[2], v[3] * t.s[3] + v[7] * t.c[3]);
    }
    return o;
}

// The lane's squares of a head.  The empty assembly makes the compiler widen x
// again where it is used next: kept from here, the fp32 values of eight heads
// would not fit the registers.
__device__ __forceinline__ float square_sum(Unit &x) {
    const float2 a = f2(x.a.x), b = f2(x.a.y), c = f2(x.b.x), d = f2(x.b.y);
    const float2 s = fma2(a, a, fma2(b, b, fma2(c, c, mul2(d, d))));
    asm volatile("" : "+r"(x.a.x), "+r"(x.a.y), "+r"(x.b.x), "+r"(x.b.y));
    return s.x + s.y;
}

// v[j], the lane's squares of its head j, becomes 1 / sqrt(mean + eps) of that
// head, which `units` lanes in a row hold (u the lane's own place among them);
// eps_of(j) is its eps.  Every lane of the warp takes part.
template <int N, class Eps>
__device__ __forceinline__ void norm_factors(float (&v)[N], float per, int units, int u, int lane, Eps eps_of) {
    if ((units & (units - 1)) == 0 && units >= N) {
        // Each step adds two lanes' sums and leaves a lane half of the heads, until
        // it holds the head whose bits, the highest first, are those of u.
        int j = 0;
#pragma unroll
        for (int n = N / 2, o = 1; n > 0; n >>= 1, o <<= 1) {
            const bool upper = (u & o) != 0;
            j += upper ? n : 0;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = upper ? v[i] : v[i + n];
                v[i] = (upper ? v[i + n] : v[i]) + __shfl_xor_sync(~0u, give, o);
            }
        }
        float sum = v[0];
        for (int o = N; o < units; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float f = rsqrtf(fmaf(sum, per, eps_of(j)));
        constexpr int kBits = N == 8 ? 3 : N == 4 ? 2 : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            int from = 0;
#pragma unroll
            for (int b = 0; b < kBits; ++b) from |= ((i >> b) & 1) << (kBits - 1 - b);
            v[i] = __shfl_sync(~0u, f, (lane & ~(N - 1)) + from);
        }
        return;
    }
    for (int o = 1; o < units; o <<= 1)  // lane u then holds the sum of lanes u .. u + 2o - 1 of its head
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float w = __shfl_down_sync(~0u, v[j], o);
            if (u + o < units) v[j] += w;
        }
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = rsqrtf(fmaf(__shfl_sync(~0u, v[j], lane - u), per, eps_of(j)));
}

// A norm's weights of the unit at `at`.
__device__ __forceinline__ Vals weights(const float *w, int2 at) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(w + at.x));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(w + at.y));
    return Vals{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The unit times its head's factor and the weights, and turned; one rounding.
__device__ __forceinline__ Unit normed(const Unit &x, float factor, const Vals &w, bool rotated, const Turn &t,
                                       int interleaved) {
    const float2 f = make_float2(factor, factor);
    const float *v = w.v;
    float2 z0 = mul2(f2(x.a.x), mul2(f, make_float2(v[0], v[1])));
    float2 z1 = mul2(f2(x.a.y), mul2(f, make_float2(v[2], v[3])));
    float2 z2 = mul2(f2(x.b.x), mul2(f, make_float2(v[4], v[5])));
    float2 z3 = mul2(f2(x.b.y), mul2(f, make_float2(v[6], v[7])));
    if (rotated) {
        if (interleaved) return turned(Vals{{z0.x, z0.y, z1.x, z1.y, z2.x, z2.y, z3.x, z3.y}}, t, 1);
        const float2 c0 = make_float2(t.c[0], t.c[1]), c1 = make_float2(t.c[2], t.c[3]);
        const float2 s0 = make_float2(t.s[0], t.s[1]), s1 = make_float2(t.s[2], t.s[3]);
        const float2 n0 = make_float2(-t.s[0], -t.s[1]), n1 = make_float2(-t.s[2], -t.s[3]);
        const float2 a0 = fma2(z2, n0, mul2(z0, c0)), a1 = fma2(z3, n1, mul2(z1, c1));
        z2 = fma2(z2, c0, mul2(z0, s0));
        z3 = fma2(z3, c1, mul2(z1, s1));
        z0 = a0;
        z1 = a1;
    }
    return Unit{make_uint2(h2(z0.x, z0.y), h2(z1.x, z1.y)), make_uint2(h2(z2.x, z2.y), h2(z3.x, z3.y))};
}

// Warp w of the grid takes heads [g * per, (g + 1) * per) of token w / groups,
// g = w % groups; lane l the unit l % units of every (32 / units)-th of them.
template <int HPL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, NORM ? kNormBlocks : kBlocks)
    rope_kernel(Heads x, Heads y, const int32_t *__restrict__ positions, Rot r, Norm n, float per, int tokens,
                int heads, FastDiv by_units, FastDiv groups) {
    pdl_wait();
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int units = by_units.d, side = 32 / by_units, sub = lane / by_units, u = lane - sub * units;
    const long long t = w / groups;
    if (t >= tokens) return;
    // (Lanes past the warp's last head help with the sums and sines, on no head.)
    const int h0 = sub < side ? w % groups * side * HPL + sub : heads;
    const int2 at = unit_parts(u, r);
    Unit v[HPL];
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        if (NORM) v[j] = Unit{make_uint2(0u, 0u), make_uint2(0u, 0u)};
        if (h0 + j * side < heads) v[j] = load_unit(x.x + t * x.token + (h0 + j * side) * x.head, at);
    }
    uint16_t *dst = const_cast<uint16_t *>(y.x) + t * y.token;
    const bool rotated = 8 * u < r.rot;
    const Turn turn = turns_of<(HPL > 1)>(r, u, units, side, sub, rotated, positions ? __ldg(positions + t) : (int)t);
    float f[HPL];
    Vals wt;
    if constexpr (NORM) {
        wt = weights(n.w, at);
#pragma unroll
        for (int j = 0; j < HPL; ++j) f[j] = square_sum(v[j]);
        norm_factors(f, per, units, u, lane, [&](int) { return n.eps; });
    }
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        if (h0 + j * side >= heads) break;
        uint16_t *out = dst + (h0 + j * side) * y.head;
        if constexpr (NORM)
            store_unit(out, at, normed(v[j], f[j], wt, rotated, turn, r.interleaved));
        else
            store_unit(out, at, rotated ? turned(vals(v[j]), turn, r.interleaved) : v[j]);
    }
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
    Rot r;
    Norm qn, kn;
    float per;  // 1 / head_dim
    int num_pages, q_heads, kv_heads;
    FastDiv page_size, units, groups;
};

// As rope_kernel, over the heads of q, then k, then v of one token; the
// token's sequence, and the page of its position, are found by the warp.
template <int HPL, bool NORM>
__global__ void __launch_bounds__(32 * kWarps, NORM ? kNormBlocks : kAppendBlocks)
    append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_wait();
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int t = w / a.groups;
    if (t >= a.b.total_q) return;
    const int units = a.units.d, side = 32 / a.units, sub = lane / a.units, u = lane - sub * units;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int h0 = w % a.groups * side * HPL + sub;
    const int2 at = unit_parts(u, a.r);
    Unit v[HPL];
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        const int h = h0 + j * side;
        if (NORM) v[j] = Unit{make_uint2(0u, 0u), make_uint2(0u, 0u)};
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
    const int slot = p % a.page_size;
    const bool rotated = 8 * u < a.r.rot;
    Turn turn;
    if (a.r.rot) turn = turns_of<(HPL > 1)>(a.r, u, units, side, sub, rotated, a.positions ? __ldg(a.positions + t) : p);
    float f[HPL];
    Vals wt;
    const float *held = nullptr;  // the norm whose weights wt holds
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < HPL; ++j) f[j] = square_sum(v[j]);
        norm_factors(f, a.per, units, u, lane, [&](int j) { return h0 + j * side < a.q_heads ? a.qn.eps : a.kn.eps; });
    }
    if (sub >= side) return;
#pragma unroll
    for (int j = 0; j < HPL; ++j) {
        const int h = h0 + j * side;
        if (h >= heads) break;
        const int hk = h - a.q_heads, hv = hk - a.kv_heads;
        if (hk >= 0 && page < 0) break;
        uint16_t *dst = hk < 0 ? a.y + t * a.y_token + h * a.y_head
                        : hv < 0 ? a.kc + page * a.kc_page + slot * a.kc_token + hk * a.kc_head
                                 : a.vc + page * a.vc_page + slot * a.vc_token + hv * a.vc_head;
        if constexpr (NORM) {
            const float *w = hk < 0 ? a.qn.w : hv < 0 ? a.kn.w : nullptr;
            if (w) {
                if (w != held) wt = weights(held = w, at);  // (a lane's heads are in the order q, k, v)
                store_unit(dst, at, normed(v[j], f[j], wt, rotated, turn, a.r.interleaved));
                continue;
            }
        }
        store_unit(dst, at, rotated && hv < 0 ? turned(vals(v[j]), turn, a.r.interleaved) : v[j]);
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

int check_norm(const f16_head_norm *n, Norm &out) {
    out = Norm{nullptr, 0.f};
    if (!n) return W4A16_OK;
    if (!n->weight) return W4_ERR_NULL;
    if (!(n->eps >= 0.f) || isinf(n->eps)) return W4_ERR_SHAPE;
    if (!aligned16(n->weight)) return W4_ERR_ALIGN;
    out = Norm{n->weight, n->eps};
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
    if (warps > 0x7FFFFFFFll - kWarps) return W4_ERR_SHAPE;
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

extern "C" int f16_rope_ex(const uint16_t *x, int64_t x_token, int64_t x_head, uint16_t *y, int64_t y_token,
                           int64_t y_head, const int32_t *positions, const f16_rotation *rotation,
                           const f16_head_norm *norm, int tokens, int heads, int head_dim, void *stream) {
    if (!rotation && !norm) return W4_ERR_NULL;
    if (tokens < 0 || heads < 1 || heads > kMaxHeads || !head_dim_ok(head_dim)) return W4_ERR_SHAPE;
    Rot r{nullptr, 0, 0, 1.f};
    Norm n;
    int st = rotation ? check_rotation(rotation, head_dim, r) : W4A16_OK;
    if (st == W4A16_OK) st = check_norm(norm, n);
    if (st != W4A16_OK) return st;
    if (tokens == 0) return W4A16_OK;
    if (!x || !y) return W4_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !stride_ok(x_token) || !stride_ok(x_head) || !stride_ok(y_token) ||
        !stride_ok(y_head) || (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
        return W4_ERR_ALIGN;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    const int units = head_dim / 8, hpl = heads_per_lane(tokens, heads, units), groups = head_groups(heads, units, hpl);
    const auto kernel = n.w ? (hpl == kManyHeads   ? rope_kernel<kManyHeads, true>
                               : hpl == kSomeHeads ? rope_kernel<kSomeHeads, true>
                                                   : rope_kernel<1, true>)
                            : (hpl == kManyHeads   ? rope_kernel<kManyHeads, false>
                               : hpl == kSomeHeads ? rope_kernel<kSomeHeads, false>
                                                   : rope_kernel<1, false>);
    return launch(kernel, (long long)tokens * groups, stream, Heads{x, x_token, x_head}, Heads{y, y_token, y_head},
                  positions, r, n, 1.f / (float)head_dim, tokens, heads, fast_div(units), fast_div(groups));
}

extern "C" int f16_rope(const uint16_t *x, int64_t x_token, int64_t x_head, uint16_t *y, int64_t y_token,
                        int64_t y_head, const int32_t *positions, const f16_rotation *rotation, int tokens, int heads,
                        int head_dim, void *stream) {
    if (!rotation) return W4_ERR_NULL;
    return f16_rope_ex(x, x_token, x_head, y, y_token, y_head, positions, rotation, nullptr, tokens, heads, head_dim,
                       stream);
}

extern "C" int f16_kv_append_ex(const uint16_t *k, int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token,
                                int64_t v_head, const f16_kv_cache *cache, const f16_kv_batch *batch,
                                const f16_rotation *rotation, const int32_t *positions, const f16_head_norm *q_norm,
                                const f16_head_norm *k_norm, const uint16_t *q, int64_t q_token, int64_t q_head,
                                uint16_t *y, int64_t y_token, int64_t y_head, int q_heads, void *stream) {
    int st = check_cache(cache);
    if (st != W4A16_OK) return st;
    AppendArgs a;
    st = check_batch(batch, cache->page_size, a.b);
    if (st != W4A16_OK) return st;
    a.r = Rot{nullptr, 0, 0, 1.f};
    if (rotation && (st = check_rotation(rotation, cache->head_dim, a.r)) != W4A16_OK) return st;
    if ((st = check_norm(q_norm, a.qn)) != W4A16_OK ||
        (st = check_norm(k_norm, a.kn)) != W4A16_OK)
        return st;
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
    a.page_size = fast_div(cache->page_size);
    a.q_heads = q ? q_heads : 0;
    a.kv_heads = cache->heads;
    const int units = cache->head_dim / 8;
    a.units = fast_div(units);
    a.per = 1.f / (float)cache->head_dim;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int hpl = heads_per_lane(batch->total_q, heads, units), groups = head_groups(heads, units, hpl);
    a.groups = fast_div(groups);
    const auto kernel = a.qn.w || a.kn.w ? (hpl == kManyHeads   ? append_kernel<kManyHeads, true>
                                            : hpl == kSomeHeads ? append_kernel<kSomeHeads, true>
                                                                : append_kernel<1, true>)
                                         : (hpl == kManyHeads   ? append_kernel<kManyHeads, false>
                                            : hpl == kSomeHeads ? append_kernel<kSomeHeads, false>
                                                                : append_kernel<1, false>);
    return launch(kernel, (long long)batch->total_q * groups, stream, a);
}

extern "C" int f16_kv_append(const uint16_t *k, int64_t k_token, int64_t k_head, const uint16_t *v, int64_t v_token,
                             int64_t v_head, const f16_kv_cache *cache, const f16_kv_batch *batch,
                             const f16_rotation *rotation, const int32_t *positions, const uint16_t *q,
                             int64_t q_token, int64_t q_head, uint16_t *y, int64_t y_token, int64_t y_head,
                             int q_heads, void *stream) {
    return f16_kv_append_ex(k, k_token, k_head, v, v_token, v_head, cache, batch, rotation, positions, nullptr, nullptr,
                            q, q_token, q_head, y, y_token, y_head, q_heads, stream);
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
