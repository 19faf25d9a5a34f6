// f16_attention for many query rows (prompts, chunks): tcgen05 tensor cores.
//
// Same mathematics as attn.cu, on tiles of 256 query rows x 128 positions.
// A unit needs 2 x 2 products of 128 x 128 x head_dim, at 4096 products a
// cycle and SM 2048 cycles for a head of 128, against 64 KB of K and V from
// L2 and 32768 exponentials, 1024 cycles at 32 a cycle: with enough rows the
// tensor cores are the bound.
//
// Measured: a prompt of 8192 tokens, 16 heads of 128 on 8, causal, 275 GFLOP:
// 222 us, 1.24 PFLOP/s, 66% of a large matrix product's rate (the tensor pipe
// busy half the time: a unit takes 3200 cycles, the chain S, softmax, P V of
// each tile).  A prompt of 1570 tokens, 16 heads on 2, 10 GFLOP: 32 us, 60000
// cycles, of which the units (four a CTA on average) take 16000 in the mean and
// 36000 where ten are left whole, plan and start 9000, parts written and joined
// through L2 (128 KB each) 8000; the rest is waiting for the slower CTAs.
// 64 tokens over 16001 positions, 66 MB of keys and values: 26 us, 22 with
// them in L2.
//
// One CTA per SM works through its range of units (attn.cuh).
//  * The item's 256 rows are two tiles of 128; tile t's scores S_t (fp32),
//    probabilities P_t (binary16) and output sums O_t (fp32) live in tensor
//    memory, one row to a lane.  While the softmax of one tile runs, the
//    tensor cores work on the other.
//  * Warps 8 and 11: copy K and V tiles page by page (tensor copies) into a ring.
//  * Warps 9 and 10: one thread for each tile issues S_t = Q_t K^T (both
//    operands in shared memory) and O_t += P_t V (P_t from tensor memory).
//    (One thread for both tiles was itself the bound, and a unit took 3850
//    cycles.)
//  * Warps 0-3 and 4-7: softmax of tile 0 and 1, one thread to a row, so row
//    sums need no exchange.  Each half of P_t is handed over as it is written,
//    so its product with V starts while the other half's exponentials are
//    taken.  (Two threads to a row, with 16 warps: no faster; tensor memory's
//    loads and stores and the agreement of the two took what was won.)
//  * Probabilities are taken against a reference that mostly stays: the
//    maximum of the row's first 64 positions.  Any reference gives the same
//    quotient o / l, and binary16 holds 2^15 with the same relative precision
//    as 1; so no unit's maximum is looked for.  Only where the sum of 64
//    probabilities passes 2^15 (none can have, up to there) is the reference
//    raised to the maximum and O_t rescaled in tensor memory.  Rounding to
//    binary16 costs a probability up to 2^-11 of itself, but nothing the one at
//    the maximum, 1; so a reference far below the maximum shows where few
//    positions take most of a row.  Items of at most 128 rows, whose softmax is
//    not what they wait for, raise it at 2^8: 64 tokens over 16001 positions
//    are 1.2 times as far from 64 bits as a plain fp32 computation (1.5 at
//    most before, now 1.3), in the same 26.5 us (at 2^6 1.1 times, 27.7 us).
//    With more rows it is 1.3 to 1.4 times (worst of 25 inputs 1.56, 24 tokens
//    over 16000); 2^8 would take 237 us, not 221, on a prompt of 8192 tokens,
//    for 1.3 times.
//  * An item of at most 128 rows has both tiles work on the same rows, one on
//    the even units, one on the odd ones; their sums are merged at its end.
//  * Positions outside a row's range get probability 0; rows of V that no row
//    of the item sees are zeroed in shared memory, as they may hold anything.
#include <math.h>
#include <string.h>

#include "attn.cuh"

namespace w4a16 {
namespace {

constexpr int QROWS = 256, KEYS = 128;
template <bool QUEUE>
using Work = Cut<QROWS, KEYS, 6, 6, 128, 10, 0, QUEUE>;
constexpr int FEW_PARTS = 4;
constexpr int QUEUE_SLOTS = 4;  // items taken ahead
constexpr int TC_THREADS = 384;
constexpr int HALF = KEYS * 128;  // bytes of 64 columns of 128 rows
// Sums of 64 probabilities past which a row's reference is raised: of an item
// of many rows 2^15, half of what binary16 holds, and of few, 2^8.
constexpr float kMostSum = 32768.f, kMostSumFew = 256.f;

template <int DP>
struct TcCfg {
    static constexpr int HALVES = DP / 64;
    static constexpr int TILE = HALVES * HALF;                    // 128 rows of Q, K or V
    static constexpr int SLOTS = DP == 64 ? 8 : 5;                // ring of K and V tiles
    static constexpr int BARS = 2 * SLOTS + 2 * 7 + 2 + 2 * QUEUE_SLOTS;
    static constexpr size_t SMEM = 1024 + (size_t)(2 + SLOTS) * TILE + 8 * BARS + 32 + 4 * QUEUE_SLOTS;
    // Tensor-memory columns.  A head of 64 leaves room for P beside S; with
    // 128, P_t lies in the columns of S_t, whose next product therefore waits
    // for O_t += P_t V to finish.
    static constexpr uint32_t S0 = 0, O0 = 256, P0 = DP == 64 ? 384 : 0, P_STEP = DP == 64 ? 64 : 128;
    static constexpr bool P_IN_S = DP != 64;
};

// Shared-memory operand descriptor: start address, leading and stride byte
// offsets, version 1, 128-byte swizzle.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((lead >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((stride >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, fp32 accumulate, binary16 operands, M = 128.
__host__ __device__ constexpr uint32_t instr_desc(int n, int b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum));
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define R8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
#define O8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
#define TMEM_LIST32                                                                                              \
    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"   \
    "%28,%29,%30,%31}"

// 32 columns of this warp's lanes; the registers hold them after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " TMEM_LIST32 ", [%32];"
                 : O8(r, 0), O8(r, 8), O8(r, 16), O8(r, 24)
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Keeps uses of r after the wait before it (no instruction).
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
    asm volatile("" : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " TMEM_LIST32 ";" ::I8(r, 0), I8(r, 8), I8(r, 16),
                 I8(r, 24), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::I8(r, 0),
        I8(r, 8), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 in one 64-bit register pair, and operations on both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(uint32_t a, uint32_t b) {
    f32x2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    return v;
}
__device__ __forceinline__ f32x2 pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 both(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
    return d;
}

// Probabilities 2^(s scale + minus) of 32 scores, rounded to binary16 in p
// and summed (unrounded) into s2.
__device__ __forceinline__ void exps(const uint32_t (&s)[32], uint32_t (&p)[16], f32x2 scale2, float minus,
                                     f32x2 (&s2)[2]) {
    const f32x2 minus2 = pair(minus, minus);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 e = both(fma2(pair(s[2 * i], s[2 * i + 1]), scale2, minus2));
        e.x = exp2_approx(e.x);
        e.y = exp2_approx(e.y);
        s2[i & 1] = add2(s2[i & 1], pair(e.x, e.y));
        p[i] = pack2(e.x, e.y);
    }
}

// Rows that a shared item's parts are stored with (4 columns of all rows
// together, [head_dim / 4][part_rows][4], so that a range of columns is one
// contiguous copy).
__device__ __forceinline__ int part_rows(int rows) { return (rows + 31) & ~31; }

// This CTA's columns of a shared item, groups of 4 from g0 to g1, by the 256
// softmax threads, a thread to a row: the parts' columns are copied into the
// ring (and their statistics over Q), as many parts at a time as fit, and
// summed in the parts' order.
template <int DP, class Sync>
__device__ __forceinline__ void join_columns(const AttnArgs &a, const Part &part, int g0, int g1, uint32_t ring,
                                             uint32_t ml_sh, uint32_t bar, uint32_t &phase, Sync sync) {
    constexpr int MOST = DP / 8;  // groups of 4 columns of one of at least two CTAs
    const int rows = part_rows(part.rows), r = threadIdx.x, ng = g1 - g0;
    const uint32_t bytes = (uint32_t)(ng * rows * 16), ml_bytes = (uint32_t)(rows * 8);
    const int most = min(TcCfg<DP>::SLOTS * TcCfg<DP>::TILE / (int)bytes, 2 * TcCfg<DP>::TILE / (QROWS * 8));
    float mx = -INFINITY, sum = 0.f;
    float4 acc[MOST];
#pragma unroll
    for (int g = 0; g < MOST; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < part.parts; p0 += most) {
        const int n = min(most, part.parts - p0);
        if (threadIdx.x == 0) {
            mbar_expect_tx(bar, n * (bytes + ml_bytes));
            for (int k = 0; k < n; ++k) {
                const long long slot = part_slot(part.first, p0 + k);
                bulk_load(ml_sh + k * ml_bytes, a.part_ml + slot * QROWS * 2, ml_bytes, bar);
                bulk_load(ring + k * bytes, a.part_o + slot * QROWS * a.head_dim + (long long)g0 * rows * 4, bytes, bar);
            }
        }
        wait(bar, phase, nullptr);
        phase ^= 1;
        if (r < part.rows) {
            for (int k = 0; k < n; ++k) {
                float2 ml;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ml.x), "=f"(ml.y) : "r"(ml_sh + k * ml_bytes + 8 * r));
                const float top = fmaxf(mx, ml.x), f0 = corr(mx, top), f1 = corr(ml.x, top);
                mx = top;
                sum = sum * f0 + ml.y * f1;
#pragma unroll
                for (int g = 0; g < MOST; ++g) {
                    if (g >= ng) break;
                    const uint4 v = lds128(ring + k * bytes + (g * rows + r) * 16);
                    acc[g].x = acc[g].x * f0 + __uint_as_float(v.x) * f1;
                    acc[g].y = acc[g].y * f0 + __uint_as_float(v.y) * f1;
                    acc[g].z = acc[g].z * f0 + __uint_as_float(v.z) * f1;
                    acc[g].w = acc[g].w * f0 + __uint_as_float(v.w) * f1;
                }
            }
        }
        fence_proxy_async_smem();  // the reads above, before the next copies
        sync();
    }
    // Out through the ring, so that lanes write neighbouring bytes of a row
    // (an odd number of 8-byte words to a row: no bank conflicts).
    const uint32_t pitch = 8 * (ng | 1);
    if (r < part.rows) {
        const float inv = inverse(sum);
#pragma unroll
        for (int g = 0; g < MOST; ++g) {
            if (g >= ng) break;
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(ring + r * pitch + 8 * g),
                         "r"(pack2(acc[g].x * inv, acc[g].y * inv)), "r"(pack2(acc[g].z * inv, acc[g].w * inv))
                         : "memory");
        }
        if (a.lse && g0 == 0) {
            const int gr = part.row0 + r, head = part.head * (int)a.group.d + gr % a.group;
            a.lse[(long long)(part.q0 + gr / a.group) * (a.kv_heads * (int)a.group.d) + head] = log_sum(mx, sum);
        }
    }
    sync();
    for (int x = threadIdx.x; x < part.rows * ng; x += 256) {
        const int row = x / ng, g = x - row * ng, gr = part.row0 + row;
        const int head = part.head * (int)a.group.d + gr % a.group;
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(ring + row * pitch + 8 * g) : "memory");
        *reinterpret_cast<uint2 *>(a.y + (part.q0 + gr / a.group) * a.y_token + head * a.y_head + 4 * (g0 + g)) = v;
    }
    fence_proxy_async_smem();  // the ring's use by threads above, before the copies of the next columns (one CTA joins all)
    sync();
}

// Block x of a shared item of many parts: 32 rows x 32 columns, a lane to a
// row, a warp to 4 columns, 16 parts' loads in flight.
__device__ __forceinline__ void join_block(const AttnArgs &a, const Part &part, int x) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col_blocks = (a.head_dim + 31) / 32, groups = a.head_dim / 4, rows = part_rows(part.rows);
    const int rb = x / col_blocks, r = 32 * rb + lane, g = 8 * (x - rb * col_blocks) + warp;
    if (r >= part.rows || g >= groups) return;
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < part.parts; i0 += 16) {
        float4 v[16];
        float2 c[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            c[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + k < part.parts) {
                const long long slot = part_slot(part.first, i0 + k);
                c[k] = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) + slot * QROWS + r);
                v[k] = __ldcg(reinterpret_cast<const float4 *>(a.part_o) + slot * groups * QROWS + g * rows + r);
            }
        }
        float top = mx;
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, c[k].x);
        const float f0 = corr(mx, top);
        mx = top;
        sum *= f0;
        acc.x *= f0;
        acc.y *= f0;
        acc.z *= f0;
        acc.w *= f0;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float f = corr(c[k].x, top);
            sum += c[k].y * f;
            acc.x += v[k].x * f;
            acc.y += v[k].y * f;
            acc.z += v[k].z * f;
            acc.w += v[k].w * f;
        }
    }
    const int gr = part.row0 + r, head = part.head * (int)a.group.d + gr % a.group;
    const long long tok = part.q0 + gr / a.group;
    const float inv = inverse(sum);
    *reinterpret_cast<uint2 *>(a.y + tok * a.y_token + head * a.y_head + 4 * g) =
        make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
    if (a.lse && g == 0) a.lse[tok * (a.kv_heads * (int)a.group.d) + head] = log_sum(mx, sum);
}

// Whether both tiles take the same rows, and alternate units.
__device__ __forceinline__ bool split_units(int rows, int n) { return rows <= 128 && n >= 2; }

// A warp's way through the CTA's pieces: those of its range, or whole items
// from a queue of all of them, the last row tiles (of causal prompts, the
// costliest) of every head and sequence first.  The warp that TAKES, the first
// to need an item, draws the CTA's next place and passes it on to the others.
// Which CTA computes an item changes nothing in it: results repeat.  (QUEUE
// false: ranges only; the code alone costs calls of few row tiles 1 us.)
template <bool QUEUE>
struct Walk : Pieces<Work<QUEUE>> {
    using Base = Pieces<Work<QUEUE>>;
    using Base::a, Base::b, Base::head, Base::left, Base::off, Base::rt, Base::s;
    uint32_t places, taken = 0, ahead;
    uint32_t bar0;               // QUEUE_SLOTS barriers each: place passed on, place read by all the other warps
    volatile uint32_t *slots;
    volatile int *abort;

    __device__ __forceinline__ Walk(const AttnArgs &args, const Plan &p, uint32_t bars, volatile uint32_t *sl, volatile int *ab)
        : Base(args, p), places(p.queue), ahead(blockIdx.x), bar0(bars), slots(sl), abort(ab) {}

    __device__ __forceinline__ bool find(uint32_t place) {  // false for one that the sequence does not have
        const uint32_t per_tile = (uint32_t)a.b.batch * a.kv_heads, back = place / per_tile, at = place - back * per_tile;
        b = (int)(at / (uint32_t)a.kv_heads);
        head = (int)(at - b * (uint32_t)a.kv_heads);
        s = load_seq(a.b, b);
        rt = row_tiles<Work<QUEUE>>(a, s) - 1 - (int)back;
        return rt >= 0;
    }
    template <bool TAKES>
    __device__ __forceinline__ bool next() {
        if (QUEUE && places != 0) {
            const int lane = threadIdx.x & 31;
            const uint32_t i = taken % QUEUE_SLOTS, phase = taken / QUEUE_SLOTS & 1;
            const uint32_t full = bar0 + 8 * i, empty = full + 8 * QUEUE_SLOTS;
            ++taken;
            uint32_t place;
            if (TAKES) {
                do {  // (the next place is on its way while this one is worked on)
                    place = uniform(ahead);
                    if (place >= places) break;
                    if (lane == 0) ahead = gridDim.x + atomicAdd(a.taken, 1u);
                } while (!find(place));
                if (!__all_sync(~0u, wait(empty, phase ^ 1, abort))) return false;
                if (lane == 0) {
                    slots[i] = place;
                    mbar_arrive(full);
                }
            } else {
                if (!__all_sync(~0u, wait(full, phase, abort))) return false;
                place = slots[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(empty);
                if (place < places) find(place);
            }
            left = place < places ? 0x40000000u : 0;  // (more than any item costs: one whole item)
            off = 0;
        }
        return Base::next();
    }
    // By one thread of the warp that takes, after its last: the last CTA of all leaves the queue as it was.
    __device__ __forceinline__ void finish() {
        if (!QUEUE || places == 0) return;
        __threadfence();
        const unsigned before = atomicAdd(a.finished, 1u);
        if (before == gridDim.x - 1) {
            if (atomicExch(a.taken, 0u) != places) atomicExch(&g_wait_expired, 1);  // (a workspace that was not zeroed)
            *a.finished = 0;
        } else if (before >= gridDim.x) {
            atomicExch(&g_wait_expired, 1);
        }
    }
};

// QUEUE: the items may come from a queue.
template <int DP, bool QUEUE>
__global__ void __launch_bounds__(TC_THREADS, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const __grid_constant__ AttnArgs a) {
    using C = TcCfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanShared plan_sh;
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t ring = base + 2 * C::TILE;
    const uint32_t bar0 = ring + C::SLOTS * C::TILE;
    uint8_t *tail = smem_raw + (bar0 - raw) + 8 * C::BARS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tail);
    volatile int *abort = reinterpret_cast<volatile int *>(tail + 4), *join_mode = abort + 1;
    volatile unsigned *seen_sh = reinterpret_cast<volatile unsigned *>(tail + 12);  // [shared item][tile]
    auto kv_full = [&](int s) { return bar0 + 8u * s; };
    auto kv_empty = [&](int s) { return bar0 + 8u * (C::SLOTS + s); };
    auto q_full = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + t); };      // Q_t written
    auto s_full = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 2 + t); };  // S_t computed
    auto o_done = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 4 + t); };  // O_t += P_t V done
    // A half (64 positions) of P_t written (and S_t read, O_t rescaled).
    auto p_full = [&](int t, int h) { return bar0 + 8u * (2 * C::SLOTS + 6 + 2 * t + h); };
    auto turn = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 10 + t); };  // tile t may issue its products
    auto o_half = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 12 + t); };  // the first half of P_t V done
    const uint32_t end_bar = bar0 + 8u * (2 * C::SLOTS + 14), join_bar = end_bar + 8, queue_bar = join_bar + 8;
    volatile uint32_t *queue_slots = reinterpret_cast<volatile uint32_t *>(tail + 28);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 2);  // both tiles' products
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full(t), 4);  // one arrival a softmax warp
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t, 0), 4);
            mbar_init(p_full(t, 1), 4);
            mbar_init(o_done(t), 1);
            mbar_init(turn(t), 1);
            mbar_init(o_half(t), 1);
        }
        mbar_init(end_bar, 2);
        mbar_init(join_bar, 1);
        *abort = 0;
        prefetch_maps(&map_k, &map_v);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (QUEUE && threadIdx.x < 32 + QUEUE_SLOTS && threadIdx.x >= 32) {
        const uint32_t at = queue_bar + 8 * (threadIdx.x - 32);
        mbar_init(at, 1);
        mbar_init(at + 8 * QUEUE_SLOTS, TC_THREADS / 32 - 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            (uint32_t)__cvta_generic_to_shared(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    constexpr int BEGINNER = 96;  // (of a warp without sequences of its own in small batches)
    Begin begin = {0, 0};
    if (threadIdx.x == BEGINNER) {
        begin = cta_begins(a);
        plan_sh.begun_before = begin.before;
    }
    fence_before();
    make_plan<Work<QUEUE>, TC_THREADS>(a, plan_sh);  // (its barriers also publish the above)
    fence_after();
    if (threadIdx.x == BEGINNER) cta_has_begun(a, begin);
    const uint32_t tmem = *tmem_slot;
    const Plan plan = plan_sh.plan;
    Walk<QUEUE> pc(a, plan, queue_bar, queue_slots, abort);

    if (warp >= 8) {
        if (warp == 8 || warp == 11) {
            // ---------------- copies: warp 8 the K tile, warp 11 the V tile of every unit, in turn ----------------
            const bool is_v = uniform(warp) == 11;
            const CUtensorMap *map = is_v ? &map_v : &map_k;
            const int boxes = KEYS / a.box_rows;  // at most 16
            int it = is_v ? 1 : 0;
            bool ok = true;
            while (ok && uniform(is_v ? pc.template next<false>() : pc.template next<true>())) {
                const int n = uniform(pc.n), head = uniform(pc.head);
                int p0 = uniform(pc.it.t0 + pc.tile0) * KEYS;
                for (int i = 0; i < n; ++i, it += 2, p0 += KEYS) {
                    const int st = it % C::SLOTS;
                    const int page = lane < boxes ? page_of(a, pc.b, p0 + lane * a.box_rows, pc.it.lo, pc.it.hi) : 0;
                    ok = __all_sync(~0u, wait(kv_empty(st), ((it / C::SLOTS) & 1) ^ 1, abort));
                    if (!ok) break;
                    const uint32_t dst = ring + st * C::TILE, bar = kv_full(st);
                    if (elect_one()) mbar_expect_tx(bar, C::TILE);
                    for (int x = 0; x < boxes; ++x) {
                        const int pg = __shfl_sync(~0u, page, x), row = x * a.box_rows;
                        if (elect_one()) {
#pragma unroll
                            for (int half = 0; half < C::HALVES; ++half)
                                tma_load_4d(dst + half * HALF + row * 128, map, 64 * half, (p0 + row) % a.page_size, head, pg,
                                            bar);
                        }
                    }
                }
            }
            if (!is_v && lane == 0) pc.finish();
            // Every copy has landed before the CTA may exit (those whose slot was taken again, by a tile up to one after
            // this warp's last, have).
            for (int k = it - 2; k >= 0 && k > it - 1 - C::SLOTS; k -= 2)
                wait(kv_full(k % C::SLOTS), (k / C::SLOTS) & 1, nullptr);
        } else if (warp < 11) {
            // ---------------- MMA issue, tile t ----------------
            // The whole warp walks the units, on values the compiler sees to
            // be the warp's and keeps in uniform registers, where the MMAs
            // take them from; one elected thread issues.
            constexpr uint32_t id_s = instr_desc(KEYS, 0), id_o = instr_desc(DP, 1);
            const int t = uniform(warp) - 9;
            const uint32_t tm = uniform(tmem);
            const uint32_t s_at = tm + C::S0 + 128 * t, p_at = tm + C::P0 + C::P_STEP * t, o_at = tm + C::O0 + DP * t;
            const uint64_t q = operand_desc(base + t * C::TILE, 16, 1024);
            int slot = 0;                          // next slot of the ring, and its phase
            uint32_t phase = 0, begun = 0, steps = 0;  // pieces begun and P V products issued
            uint32_t turns = 0;                        // steps of pieces with both tiles
            bool ok = true;
            auto advance = [&] {
                if (++slot == C::SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            auto await = [&](uint32_t bar, uint32_t parity) { ok = __all_sync(~0u, ok && wait(bar, parity, abort)); };
            auto score = [&](int at) {  // S = Q K^T, K in slot `at`
                const uint64_t kt = operand_desc(ring + at * C::TILE, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s) {  // 16 columns: 32 bytes on, or the next 64 columns
                        const uint32_t off = ((s / 4) * HALF + (s % 4) * 32) >> 4;
                        mma_ss(s_at, q + off, kt + off, id_s, s != 0);
                    }
                    commit(s_full(t));
                    commit(kv_empty(at));
                }
            };
            while (ok && uniform(pc.template next<false>())) {
                const int n = uniform(pc.n), rows = uniform(pc.rows());
                const bool split = split_units(rows, n), both_tiles = rows > 128;
                auto hand_on = [&](int slots) {  // slots that this tile does not use
                    for (int i = 0; ok && i < slots; ++i) {
                        await(kv_full(slot), phase);
                        if (ok && elect_one()) mbar_arrive(kv_empty(slot));
                        advance();
                    }
                };
                if (128 * t >= rows && !split) {
                    hand_on(2 * n);
                    continue;
                }
                const int stride = split ? 2 : 1;
                if (split && t) hand_on(2);
                await(q_full(t), begun++ & 1);
                await(kv_full(slot), phase);
                // the columns of S, if P lies there: the last product of the piece before has read it
                if (C::P_IN_S && steps > 0) await(o_done(t), (steps - 1) & 1);
                if (!ok) break;
                fence_after();
                score(slot);
                advance();
                bool first = true;
                for (int j = split ? t : 0; j < n; j += stride) {
                    const int v_slot = slot;
                    const bool more = j + stride < n;
                    // K of the next unit too, ahead of the probabilities
                    await(kv_full(slot), phase);
                    advance();
                    if (more && !split) await(kv_full(slot), phase);
                    const uint64_t vt = operand_desc(ring + v_slot * C::TILE, HALF, 1024);
                    if (both_tiles) await(turn(t), (turns++ & 1) ^ (t == 0 ? 1 : 0));
                    await(p_full(t, 0), steps & 1);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) mma_ts(o_at, p_at + 8 * s, vt + s * (2048 >> 4), id_o, !first || s != 0);
                        commit(o_half(t));
                    }
                    first = false;
                    await(p_full(t, 1), steps & 1);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 4; s < 8; ++s) mma_ts(o_at, p_at + 8 * s, vt + s * (2048 >> 4), id_o, 1);
                        commit(o_done(t));
                        commit(kv_empty(v_slot));
                    }
                    // The next K, past the other tile's unit in between.
                    const int skip = split ? 2 : 0;
                    const bool wraps = slot + skip >= C::SLOTS;
                    const int k_slot = wraps ? slot + skip - C::SLOTS : slot + skip;
                    if (more) {
                        if (split) await(kv_full(k_slot), phase ^ (wraps ? 1 : 0));
                        if (C::P_IN_S) await(o_done(t), steps & 1);
                        if (!ok) break;
                    }
                    // The other tile's products may queue up behind this one's last.
                    if (both_tiles && elect_one()) mbar_arrive(turn(t ^ 1));
                    if (more) score(k_slot);
                    if (split && j + 1 < n) hand_on(2);
                    if (more) advance();
                    ++steps;
                }
            }
            if (elect_one()) commit(end_bar);  // every product is done before the CTA may exit
            wait(end_bar, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ---------------- softmax: warps 4 t .. 4 t + 3 for tile t, one thread to a row ----------------
        const int t = warp >> 2, quad = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_at = lanes + C::S0 + 128 * t, p_at = lanes + C::P0 + C::P_STEP * t, o_at = lanes + C::O0 + DP * t;
        // Row rl of this warp's 32 rows of Q_t, 16-byte chunk ch (also the way out of y's rows).
        const uint32_t my_rows = base + t * C::TILE + 32 * quad * 128;
        auto stage_at = [&](int rl, int ch) { return my_rows + (ch / 8) * HALF + rl * 128 + (((ch ^ rl) & 7) << 4); };
        const f32x2 scale2 = pair(a.scale, a.scale);
        Part shared0, shared1;  // items that this CTA shares with earlier and later ones
        int shares = 0;
        bool uncounted = false;  // this thread has a part to count in
        bool waits = true;       // and whether it may wait for the others'
        uint32_t steps = 0;
        int it = 0;
        while (pc.template next<false>()) {
            const int first_slot = it;
            it += 2 * pc.n;
            const int rows = pc.rows(), row0 = pc.row0();
            const bool whole = pc.begins && pc.ends;
            auto note_part = [&] {
                if (whole) return;
                if (shares++ == 0)
                    shared0 = pc.part(plan);
                else
                    shared1 = pc.part(plan);
            };
            auto count_first = [&] {  // (of the first shared item: a later one is this CTA's last)
                if (uncounted) seen_sh[t] = count_part<true>(a, shared0, plan_sh.begun_before, waits);
                uncounted = false;
            };
            const bool split = split_units(rows, pc.n);
            const int tile_row = split ? 0 : 128 * t;
            if (tile_row >= rows) {
                count_first();
                note_part();
                continue;
            }
            const int r = tile_row + 32 * quad + lane;  // this thread's row of the item
            const bool in = r < rows;
            const int gr = row0 + r;
            const long long tok = pc.s.q0 + gr / a.group;
            const int head = pc.head * (int)a.group.d + gr % a.group;
            // Q_t: the warp's 32 rows, 16 bytes a lane, swizzled, all in flight together.
            // Four lanes take 64 bytes of a row, 8 rows at a time: a row's address is needed once.
            const long long q_row = in ? tok * a.q_token + head * a.q_head : -1;
#pragma unroll
            for (int rb = 0; rb < 32; rb += 8) {
                const int rl = rb + (lane >> 2);
                const long long at = __shfl_sync(~0u, q_row, rl);
                const uint16_t *src = a.q + (at >= 0 ? at : 0) + 8 * (lane & 3);
#pragma unroll
                for (int c4 = 0; c4 < DP / 8; c4 += 4) {
                    const int ch = c4 + (lane & 3);
                    const bool has = at >= 0 && 8 * ch < a.head_dim;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(stage_at(rl, ch)),
                                 "l"(has ? src + 8 * c4 : a.q), "r"(has ? 16 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full(t));
            count_first();  // now that there is time, until S_t is there
            note_part();

            const int p = pc.s.kv - pc.s.qn + gr / a.group;
            const int ub = in ? (a.causal ? min(p + 1, pc.s.kv) : pc.s.kv) : 0;
            const int lb = a.window > 0 ? p - a.window + 1 : 0;
            // Units inside these bounds need no mask for any row of the tile.
            const int pf = pc.s.kv - pc.s.qn + (row0 + tile_row) / a.group;
            const int pl = pc.s.kv - pc.s.qn + (row0 + min(rows, tile_row + 128) - 1) / a.group;
            const int all_ub = a.causal ? min(pf + 1, pc.s.kv) : pc.s.kv;
            const int all_lb = a.window > 0 ? pl - a.window + 1 : 0;

            // Reference (of scores in base 2) and sum.  (Rows past the item's end see nothing and need no reference.)
            float ref = in ? -INFINITY : 0.f, sum = 0.f;
            const int j_first = split ? t : 0;
            for (int j = j_first; j < pc.n; j += split ? 2 : 1, ++steps) {
                const int j0 = (pc.it.t0 + pc.tile0 + j) * KEYS;
                wait(s_full(t), steps & 1, abort);
                fence_after();
                if (j0 + KEYS > all_ub || j0 < all_lb) {  // positions that not every row sees: scores to -infinity
#pragma unroll 1
                    for (int c = 0; c < KEYS; c += 32) {
                        const int lo = lb - j0 - c, hi = ub - j0 - c;
                        uint32_t v[32];
                        tmem_load(s_at + c, v);
                        tmem_load_wait();
                        tmem_loaded(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (i < lo || i >= hi) v[i] = 0xFF800000u;
                        tmem_store(s_at + c, v);
                    }
                    tmem_store_wait();
                }
                if (j0 < pc.it.lo || j0 + KEYS > pc.it.hi) {
                    // Rows of V that the item does not see: one to a thread (both tiles write the same zeros, each
                    // before its own product).
                    const int k = first_slot + 2 * j + 1, row = 32 * quad + lane;
                    wait(kv_full(k % C::SLOTS), (k / C::SLOTS) & 1, abort);
                    if (j0 + row < pc.it.lo || j0 + row >= pc.it.hi) {
#pragma unroll
                        for (int x = 0; x < DP / 8; ++x)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             ring + k % C::SLOTS * C::TILE + (x / 8) * HALF + row * 128 + (x % 8) * 16),
                                         "r"(0)
                                         : "memory");
                    }
                    fence_proxy_async_smem();
                }
                // (Loops kept short where they can be: the warps' code is fetched anew every time round.)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t sr[2][32], pr[2][16];
                    tmem_load(s_at + 64 * h, sr[0]);
                    tmem_load(s_at + 64 * h + 32, sr[1]);
                    tmem_load_wait();
                    tmem_loaded(sr[0]);
                    tmem_loaded(sr[1]);
                    float part_sum;
#pragma unroll 1
                    for (bool again = false;; again = true) {
                        f32x2 s2[2] = {0, 0};
                        const float minus = ref == -INFINITY ? 0.f : -ref;
                        exps(sr[0], pr[0], scale2, minus, s2);
                        exps(sr[1], pr[1], scale2, minus, s2);
                        const float2 e = both(add2(s2[0], s2[1]));
                        part_sum = e.x + e.y;
                        const bool raise = !(part_sum <= (split ? kMostSumFew : kMostSum)) || ref == -INFINITY;
                        if (again || !__any_sync(~0u, raise)) break;
                        float m = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 32; ++i) m = max3(m, sr[0][i], sr[1][i]);
                        const float nr = raise ? fmaxf(ref, m * a.scale) : ref;
                        const float c = nr != ref ? corr(ref, nr) : 1.f;
                        if (j > j_first || h > 0) {  // O_t holds something
                            wait(h ? o_half(t) : o_done(t), (h ? steps : steps - 1) & 1, abort);
                            fence_after();
#pragma unroll 1
                            for (int cb = 0; cb < DP / 32; ++cb) {
                                uint32_t o[32];
                                tmem_load(o_at + 32 * cb, o);
                                tmem_load_wait();
                                tmem_loaded(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * c);
                                tmem_store(o_at + 32 * cb, o);
                            }
                            tmem_store_wait();
                        }
                        sum *= c;
                        ref = nr;
                    }
                    sum += part_sum;
                    tmem_store16(p_at + 32 * h, pr[0]);
                    tmem_store16(p_at + 32 * h + 16, pr[1]);
                    tmem_store_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(t, h));
                }
            }

            // ---------------- the piece's rows ----------------
            wait(o_done(t), (steps - 1) & 1, abort);
            fence_after();
            const uint32_t other = base + C::TILE;  // over Q_1
            float f0 = 1.f, f1 = 0.f;
            auto both_sync = [] { asm volatile("bar.sync 4, 256;" ::: "memory"); };
            if (split) {  // tile 0 gets tile 1's reference and sum, then its outputs 32 columns at a time
                const uint32_t at = other + 8 * (32 * quad + lane);
                if (t) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(ref), "f"(sum) : "memory");
                both_sync();
                if (!t) {
                    float2 v;
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
                    const float top = fmaxf(ref, v.x);
                    f0 = corr(ref, top);
                    f1 = corr(v.x, top);
                    ref = top;
                    sum = sum * f0 + v.y * f1;
                }
                both_sync();
            }
            if (in && !(split && t)) {
                if (!whole)
                    reinterpret_cast<float2 *>(a.part_ml)[(long long)pc.slot() * QROWS + r] = make_float2(ref, sum);
                else if (a.lse)
                    a.lse[tok * (a.kv_heads * (int)a.group.d) + head] = log_sum(ref, sum);
            }
            const float inv = inverse(sum);
            float4 *part = reinterpret_cast<float4 *>(a.part_o) + (long long)pc.slot() * QROWS * (a.head_dim / 4) + r;
            const int p_rows = part_rows(rows);
#pragma unroll 1
            for (int cb = 0; cb < DP / 32; ++cb) {
                uint32_t o[32];
                tmem_load(o_at + 32 * cb, o);
                tmem_load_wait();
                tmem_loaded(o);
                if (split) {
                    const uint32_t at = other + 4 * (32 * quad + lane);
                    if (t) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 512 * i), "r"(o[i]) : "memory");
                    }
                    both_sync();
                    if (!t) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            float v;
                            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at + 512 * i));
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f0 + v * f1);
                        }
                    }
                    both_sync();
                    if (t) continue;
                }
                if (whole) {  // through this warp's rows of Q_t (its products are done)
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = pack2(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage_at(lane, 4 * cb + i / 8)),
                                     "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                                     : "memory");
                    }
                } else if (in) {  // 4 columns of all rows lie together
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (32 * cb + i < a.head_dim)
                            part[(8 * cb + i / 4) * p_rows] =
                                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                            __uint_as_float(o[i + 3]));
                }
            }
            if (whole && !(split && t)) {
                __syncwarp();
                const long long y_row = in ? tok * a.y_token + head * a.y_head : -1;
#pragma unroll
                for (int rb = 0; rb < 32; rb += 8) {
                    const int rl = rb + (lane >> 2);
                    const long long at = __shfl_sync(~0u, y_row, rl);
                    uint4 v[DP / 32];
#pragma unroll
                    for (int k = 0; k < DP / 32; ++k) v[k] = lds128(stage_at(rl, 4 * k + (lane & 3)));
#pragma unroll
                    for (int k = 0; k < DP / 32; ++k) {
                        const int ch = 4 * k + (lane & 3);
                        if (at >= 0 && 8 * ch < a.head_dim) *reinterpret_cast<uint4 *>(a.y + at + 8 * ch) = v[k];
                    }
                }
                __syncwarp();
            }
            fence_before();  // the reads above, before the next piece's first product writes O_t
            if (!whole && !(split && t)) {
                if (t == 0)  // this tile's warps
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                else
                    asm volatile("bar.sync 2, 128;" ::: "memory");
                uncounted = (threadIdx.x & 127) == 0;
            }
        }
        // ---------------- join this CTA's share of the items it shares, all eight warps ----------------
        // (Both tiles' warps meet before the first copy into the ring: every product is done.)
        if (uncounted) seen_sh[2 * (shares - 1) + t] = count_part<true>(a, shares == 1 ? shared0 : shared1, plan_sh.begun_before, waits);
        uint32_t join_phase = 0;
        for (int i = 0; i < shares; ++i) {
            const Part part = i == 0 ? shared0 : shared1;
            auto sync = [] { asm volatile("bar.sync 3, 256;" ::: "memory"); };
            // Few parts: ranges of columns, by copies, some 26 bytes a cycle where loads of the same parts ran at 17
            // (a prompt of 1570 tokens: 33 us, against 43 by blocks).  Many: blocks of rows
            // and columns, as a joiner's range of columns would be a few bytes.
            const bool few = part.parts <= FEW_PARTS;
            const int groups = a.head_dim / 4, blocks = (part.rows + 31) / 32 * ((a.head_dim + 31) / 32);
            const int joiners = min(part.parts, few ? groups : blocks);
            fence_proxy_async_smem();  // (shared memory that threads used is written by copies)
            sync();
            if (threadIdx.x == 0) {
                // The later of the counts that the tiles' threads saw.  (A CTA with no share need not wait.)
                const unsigned tiles = part.rows > 128 ? 2 : 1, all = part.parts * tiles;
                const unsigned s0 = seen_sh[2 * i], s1 = tiles == 2 ? seen_sh[2 * i + 1] : 0;
                const unsigned seen = (s1 & kCountMask) > (s0 & kCountMask) ? s1 : s0;
                *join_mode = await_parts(a, part, seen, part.index < joiners && waits, all);
                asm volatile("fence.proxy.async.global;" ::: "memory");  // the parts were stored by threads, and are read by copies
            }
            sync();
            const int mode = *join_mode;
            // Columns are one range to a joiner, blocks are dealt out in turn.
            const int pieces = few ? joiners : blocks;
            const int step = mode == kJoinAll ? 1 : joiners;
            for (int x = mode == kJoinAll ? 0 : part.index; mode != kJoinNothing && x < pieces; x += step) {
                if (few)
                    join_columns<DP>(a, part, x * groups / joiners, (x + 1) * groups / joiners, ring, base, join_bar,
                                     join_phase, sync);
                else
                    join_block(a, part, x);
            }
            sync();
            if (threadIdx.x == 0) part_done(a, part);
        }
    }

    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <int DP, bool QUEUE>
int launch_tc(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    static_assert(TcCfg<DP>::SMEM + sizeof(PlanShared) <= 227 * 1024, "shared memory");
    if (!ensure_smem(reinterpret_cast<const void *>(attn_tc_kernel<DP, QUEUE>), TcCfg<DP>::SMEM)) return W4_ERR_LAUNCH;
    return launch_dependent(attn_tc_kernel<DP, QUEUE>, grid, TC_THREADS, TcCfg<DP>::SMEM, stream, mk, mv, a);
}

}  // namespace

int attn_tc_rows() { return QROWS; }

int attn_tc_launch(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    if (a.head_dim <= 64)
        return a.may_queue ? launch_tc<64, true>(mk, mv, a, grid, stream) : launch_tc<64, false>(mk, mv, a, grid, stream);
    return a.may_queue ? launch_tc<128, true>(mk, mv, a, grid, stream) : launch_tc<128, false>(mk, mv, a, grid, stream);
}

// This translation unit's records, as attn_status.
int attn_tc_status() {
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
