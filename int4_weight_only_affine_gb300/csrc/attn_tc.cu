// f16_attention for many query rows (prompts, chunks): tcgen05 tensor cores.
//
// Same mathematics as attn.cu, on tiles of 256 query rows x 128 positions.
// A unit needs 2 x 2 products of 128 x 128 x head_dim, at 4096 products a
// cycle and SM 2048 cycles for a head of 128, against 64 KB of K and V from
// L2 and 32768 exponentials: with enough rows the tensor cores are the bound.
//
// One CTA per SM works through its range of units (attn.cuh).
//  * The item's 256 rows are two tiles of 128; tile t's scores S_t (fp32),
//    probabilities P_t (binary16) and output sums O_t (fp32) live in tensor
//    memory, one row to a lane.  While the softmax of one tile runs, the
//    tensor cores work on the other.
//  * Warps 8 and 11: copy K and V tiles page by page (tensor copies) into a ring.
//  * Warps 9 and 10: one thread for each tile issues S_t = Q_t K^T (both
//    operands in shared memory) and O_t += P_t V (P_t from tensor memory).
//    (One thread for both tiles was itself the bound: 3850 cycles a unit.)
//  * Warps 0-3 and 4-7: softmax of tile 0 and 1, one thread to a row, so row
//    maxima and sums need no exchange.  Each half of P_t is handed over as it
//    is written, so its product with V starts while the other half's
//    exponentials are taken.  O_t is rescaled in tensor memory only
//    when a row's maximum has grown by more than 2^8 since the last time:
//    until then probabilities are taken against the older maximum, which
//    makes them at most 256 and changes nothing else (the quotient o / l does
//    not depend on the reference; binary16 holds 256 with the same relative
//    precision as 1).
//  * Positions outside a row's range get probability 0; rows of V that no row
//    of the item sees are zeroed in shared memory, as they may hold anything.
#include <math.h>
#include <string.h>

#include "attn.cuh"

namespace w4a16 {
namespace {

constexpr int QROWS = 256, KEYS = 128;
constexpr int TC_THREADS = 384;
// Registers a thread: 168 at launch (64512 in all); the softmax's two warp
// groups take what the third (copies, MMA issue) gives up.
constexpr int REGS_LAUNCH = 168, REGS_SOFTMAX = 208, REGS_OTHER = 88;
static_assert(2 * REGS_SOFTMAX + REGS_OTHER == 3 * REGS_LAUNCH, "register split");
constexpr int HALF = KEYS * 128;  // bytes of 64 columns of 128 rows
constexpr float kGrow = 8.f;      // growth of the maximum (base 2) that rescales

template <int DP>
struct TcCfg {
    static constexpr int HALVES = DP / 64;
    static constexpr int TILE = HALVES * HALF;                    // 128 rows of Q, K or V
    static constexpr int SLOTS = DP == 64 ? 8 : 5;                // ring of K and V tiles
    static constexpr int BARS = 2 * SLOTS + 2 * 6 + 1;
    static constexpr size_t SMEM = 1024 + (size_t)(2 + SLOTS) * TILE + 8 * BARS + 16;
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

// mbar_wait without a call: the register split leaves no room for one.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    uint64_t t0 = 0;  // the clock is read only once a wait has become long
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

// Scores of positions 32 C .. 32 C + 31 of a unit: those outside [lo, hi) to
// -infinity, maxima of the others into m4.
template <int C>
__device__ __forceinline__ void mask_and_max(uint32_t (&s)[32], float (&m4)[4], bool masked, int lo, int hi) {
    if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (32 * C + i < lo || 32 * C + i >= hi) s[i] = 0xFF800000u;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) m4[i / 2 % 4] = max3(m4[i / 2 % 4], s[i], s[i + 1]);
}

template <int DP>
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
    volatile int *abort = reinterpret_cast<volatile int *>(tail + 4);
    auto kv_full = [&](int s) { return bar0 + 8u * s; };
    auto kv_empty = [&](int s) { return bar0 + 8u * (C::SLOTS + s); };
    auto q_full = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + t); };      // Q_t written
    auto s_full = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 2 + t); };  // S_t computed
    auto o_done = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 4 + t); };  // O_t += P_t V done
    // A half (64 positions) of P_t written (and S_t read, O_t rescaled).
    auto p_full = [&](int t, int h) { return bar0 + 8u * (2 * C::SLOTS + 6 + 2 * t + h); };
    auto turn = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 10 + t); };  // tile t may issue its products
    const uint32_t end_bar = bar0 + 8u * (2 * C::SLOTS + 12);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
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
        }
        mbar_init(end_bar, 2);
        *abort = 0;
        a.joins[blockIdx.x].parts = 0;
        prefetch_maps(&map_k, &map_v);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
            (uint32_t)__cvta_generic_to_shared(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    make_plan<QROWS, KEYS, TC_THREADS, 1>(a, plan_sh);  // (its barriers also publish the above)
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const Plan plan = plan_sh.plan;
    Pieces<QROWS, KEYS> pc(a, plan);

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
        if (warp == 8 || warp == 11) {
            // ---------------- copies: warp 8 the K tile, warp 11 the V tile of every unit, in turn ----------------
            const bool is_v = uniform(warp) == 11;
            const CUtensorMap *map = is_v ? &map_v : &map_k;
            const int boxes = KEYS / a.box_rows;  // at most 16
            int it = is_v ? 1 : 0;
            bool ok = true;
            while (ok && uniform(pc.next())) {
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
            auto score = [&] {  // S = Q K^T, K in the next slot
                const uint64_t kt = operand_desc(ring + slot * C::TILE, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s) {  // 16 columns: 32 bytes on, or the next 64 columns
                        const uint32_t off = ((s / 4) * HALF + (s % 4) * 32) >> 4;
                        mma_ss(s_at, q + off, kt + off, id_s, s != 0);
                    }
                    commit(s_full(t));
                    commit(kv_empty(slot));
                }
                advance();
            };
            while (ok && uniform(pc.next())) {
                const int n = uniform(pc.n), rows = uniform(pc.rows());
                if (128 * t >= rows) {  // no such tile: only hand the slots on
                    for (int i = 0; ok && i < 2 * n; ++i) {
                        await(kv_full(slot), phase);
                        if (ok && elect_one()) mbar_arrive(kv_empty(slot));
                        advance();
                    }
                    continue;
                }
                await(q_full(t), begun++ & 1);
                await(kv_full(slot), phase);
                // the columns of S, if P lies there: the last product of the piece before has read it
                if (C::P_IN_S && steps > 0) await(o_done(t), (steps - 1) & 1);
                if (!ok) break;
                fence_after();
                score();
                const bool both_tiles = rows > 128;
                for (int j = 0; j < n; ++j) {
                    const int v_slot = slot;
                    const bool more = j + 1 < n;
                    // K of the next unit too, ahead of the probabilities
                    await(kv_full(slot), phase);
                    advance();
                    if (more) await(kv_full(slot), phase);
                    const uint64_t vt = operand_desc(ring + v_slot * C::TILE, HALF, 1024);
                    if (both_tiles) await(turn(t), (turns++ & 1) ^ (t == 0 ? 1 : 0));
                    await(p_full(t, 0), steps & 1);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) mma_ts(o_at, p_at + 8 * s, vt + s * (2048 >> 4), id_o, (j | s) != 0);
                    }
                    await(p_full(t, 1), steps & 1);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 4; s < 8; ++s) mma_ts(o_at, p_at + 8 * s, vt + s * (2048 >> 4), id_o, 1);
                        commit(o_done(t));
                        commit(kv_empty(v_slot));
                    }
                    if (more) {
                        if (C::P_IN_S) await(o_done(t), steps & 1);
                        if (!ok) break;
                    }
                    // The other tile's products may queue up behind this one's last.
                    if (both_tiles && elect_one()) mbar_arrive(turn(t ^ 1));
                    if (more) score();
                    ++steps;
                }
            }
            if (elect_one()) commit(end_bar);  // every product is done before the CTA may exit
            wait(end_bar, 0, nullptr);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        // ---------------- softmax: warps 4 t .. 4 t + 3 for tile t, one thread to a row ----------------
        const int t = warp >> 2, quad = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_at = lanes + C::S0 + 128 * t, p_at = lanes + C::P0 + C::P_STEP * t, o_at = lanes + C::O0 + DP * t;
        // Row rl of this warp's 32 rows of Q_t, 16-byte chunk ch (also the way out of y's rows).
        const uint32_t my_rows = base + t * C::TILE + 32 * quad * 128;
        auto stage_at = [&](int rl, int ch) { return my_rows + (ch / 8) * HALF + rl * 128 + (((ch ^ rl) & 7) << 4); };
        const f32x2 scale2 = pair(a.scale, a.scale);
        uint32_t steps = 0;
        int it = 0;
        while (pc.next()) {
            const int first_slot = it;
            it += 2 * pc.n;
            const int rows = pc.rows(), row0 = pc.row0();
            if (128 * t >= rows) continue;
            const int r = 128 * t + 32 * quad + lane;  // this thread's row of the item
            const bool in = r < rows;
            const int gr = row0 + r;
            const long long tok = pc.s.q0 + gr / a.group;
            const int head = pc.head * (int)a.group.d + gr % a.group;
            // Q_t: the warp's 32 rows, 16 bytes a lane, swizzled, all in flight together.
            const long long q_row = in ? tok * a.q_token + head * a.q_head : -1;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
                const int x = 32 * i + lane, rl = x / (DP / 8), ch = x % (DP / 8);
                const long long at = __shfl_sync(~0u, q_row, rl);
                const bool has = at >= 0 && 8 * ch < a.head_dim;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(stage_at(rl, ch)),
                             "l"(has ? a.q + at + 8 * ch : a.q), "r"(has ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full(t));

            const int p = pc.s.kv - pc.s.qn + gr / a.group;
            const int ub = in ? (a.causal ? min(p + 1, pc.s.kv) : pc.s.kv) : 0;
            const int lb = a.window > 0 ? p - a.window + 1 : 0;
            // Units inside these bounds need no mask for any row of the tile.
            const int pf = pc.s.kv - pc.s.qn + (row0 + 128 * t) / a.group;
            const int pl = pc.s.kv - pc.s.qn + (row0 + min(rows, 128 * t + 128) - 1) / a.group;
            const int all_ub = a.causal ? min(pf + 1, pc.s.kv) : pc.s.kv;
            const int all_lb = a.window > 0 ? pl - a.window + 1 : 0;

            float ref = -INFINITY, sum = 0.f;  // reference maximum (base-2 scaled scores) and sum
            for (int j = 0; j < pc.n; ++j, ++steps) {
                const int j0 = (pc.it.t0 + pc.tile0 + j) * KEYS;
                wait(s_full(t), steps & 1, abort);
                fence_after();
                uint32_t sr[4][32];
                tmem_load(s_at, sr[0]);
                tmem_load(s_at + 32, sr[1]);
                tmem_load_wait();
                tmem_load(s_at + 64, sr[2]);
                tmem_load(s_at + 96, sr[3]);
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const bool masked = j0 + KEYS > all_ub || j0 < all_lb;
                const int lo = lb - j0, hi = ub - j0;
                tmem_loaded(sr[0]);
                tmem_loaded(sr[1]);
                mask_and_max<0>(sr[0], m4, masked, lo, hi);
                mask_and_max<1>(sr[1], m4, masked, lo, hi);
                tmem_load_wait();
                tmem_loaded(sr[2]);
                tmem_loaded(sr[3]);
                mask_and_max<2>(sr[2], m4, masked, lo, hi);
                mask_and_max<3>(sr[3], m4, masked, lo, hi);
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale;
                const bool grow = mx > ref + kGrow || (ref == -INFINITY && mx > ref);
                if (__any_sync(~0u, grow)) {
                    const float nr = grow ? mx : ref;
                    const float c = ref == -INFINITY ? 0.f : exp2_approx(ref - nr);
                    if (j > 0) {
                        wait(o_done(t), (steps - 1) & 1, abort);
                        fence_after();
#pragma unroll 1
                        for (int cb = 0; cb < DP / 32; ++cb) {
                            uint32_t o[32];
                            tmem_load(o_at + 32 * cb, o);
                            tmem_load_wait();
                            tmem_loaded(o);
                            const float f = grow ? c : 1.f;
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_store(o_at + 32 * cb, o);
                        }
                        tmem_store_wait();
                    }
                    if (grow) {
                        sum *= c;
                        ref = nr;
                    }
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
                const float minus = ref == -INFINITY ? 0.f : -ref;
                const f32x2 minus2 = pair(minus, minus);
                f32x2 s2[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pr[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 e = both(fma2(pair(sr[c][2 * i], sr[c][2 * i + 1]), scale2, minus2));
                        e.x = exp2_approx(e.x);
                        e.y = exp2_approx(e.y);
                        s2[i & 1] = add2(s2[i & 1], pair(e.x, e.y));
                        pr[i] = pack2(e.x, e.y);
                    }
                    tmem_store16(p_at + 16 * c, pr);
                    if (c & 1) {
                        tmem_store_wait();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_full(t, c >> 1));
                    }
                }
                const float2 s4 = both(add2(s2[0], s2[1]));
                sum += s4.x + s4.y;
            }

            // ---------------- the piece's rows ----------------
            wait(o_done(t), (steps - 1) & 1, abort);
            fence_after();
            const bool whole = pc.begins && pc.ends;
            if (in) {
                if (!whole)
                    reinterpret_cast<float2 *>(a.part_ml)[(long long)pc.slot() * QROWS + r] = make_float2(ref, sum);
                else if (a.lse)
                    a.lse[tok * (a.kv_heads * (int)a.group.d) + head] = log_sum(ref, sum);
            }
            if (threadIdx.x == 0 && pc.begins && !pc.ends)
                a.joins[blockIdx.x] = JoinItem{pc.parts(plan), pc.s.q0, pc.head, row0, rows};
            const float inv = inverse(sum);
            float4 *part = reinterpret_cast<float4 *>(a.part_o) + (long long)pc.slot() * QROWS * (a.head_dim / 4) + r;
#pragma unroll 1
            for (int cb = 0; cb < DP / 32; ++cb) {
                uint32_t o[32];
                tmem_load(o_at + 32 * cb, o);
                tmem_load_wait();
                tmem_loaded(o);
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
                            part[(8 * cb + i / 4) * QROWS] =
                                make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                            __uint_as_float(o[i + 3]));
                }
            }
            if (whole) {
                __syncwarp();
                const long long y_row = in ? tok * a.y_token + head * a.y_head : -1;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) {
                    const int x = 32 * i + lane, rl = x / (DP / 8), ch = x % (DP / 8);
                    const long long at = __shfl_sync(~0u, y_row, rl);
                    if (at >= 0 && 8 * ch < a.head_dim) *reinterpret_cast<uint4 *>(a.y + at + 8 * ch) = lds128(stage_at(rl, ch));
                }
                __syncwarp();
            }
            fence_before();  // the reads above, before the next piece's first product writes O_t
        }
    }

    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// Join of the items that attn_tc_kernel cut: block (c, n) joins rows 32 n ..
// 32 n + 31 of the item that starts in the range of CTA c, a lane to a row, a
// warp to every 8th group of 4 columns.
constexpr int JOIN_WARPS = 8;
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_tc_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ __align__(16) uint16_t out[32][128 + 8];
    pdl_wait();
    const JoinItem j = a.joins[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = 32 * blockIdx.y + lane;
    if (32 * (int)blockIdx.y >= j.rows || j.parts == 0) return;
    const int groups = a.head_dim / 4;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + r;
    const float4 *po = reinterpret_cast<const float4 *>(a.part_o) + r;
    float mx = -INFINITY, sum = 0.f;
    float4 acc[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < j.rows) {
        for (int i0 = 0; i0 < j.parts; i0 += 4) {  // four parts' loads in flight
            float4 v[4][4];
            float2 c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c[k] = make_float2(-INFINITY, 0.f);
                if (i0 + k < j.parts) {
                    const long long slot = part_slot(blockIdx.x, i0 + k);
                    c[k] = ml[slot * QROWS];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (warp + JOIN_WARPS * g < groups) v[k][g] = po[(slot * groups + warp + JOIN_WARPS * g) * QROWS];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i0 + k >= j.parts) break;
                const float top = fmaxf(mx, c[k].x), f0 = corr(mx, top), f1 = corr(c[k].x, top);
                mx = top;
                sum = sum * f0 + c[k].y * f1;
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    if (warp + JOIN_WARPS * g < groups) {
                        acc[g].x = acc[g].x * f0 + v[k][g].x * f1;
                        acc[g].y = acc[g].y * f0 + v[k][g].y * f1;
                        acc[g].z = acc[g].z * f0 + v[k][g].z * f1;
                        acc[g].w = acc[g].w * f0 + v[k][g].w * f1;
                    }
            }
        }
        const float inv = inverse(sum);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (warp + JOIN_WARPS * g < groups)
                *reinterpret_cast<uint2 *>(&out[lane][4 * (warp + JOIN_WARPS * g)]) =
                    make_uint2(pack2(acc[g].x * inv, acc[g].y * inv), pack2(acc[g].z * inv, acc[g].w * inv));
        if (a.lse && warp == 0) {
            const int gr = j.row0 + r;
            a.lse[(long long)(j.q0 + gr / a.group) * (a.kv_heads * (int)a.group.d) + j.head * (int)a.group.d +
                  gr % a.group] = log_sum(mx, sum);
        }
    }
    __syncthreads();
    const int chunks = a.head_dim / 8;
    for (int x = threadIdx.x; x < 32 * chunks; x += 32 * JOIN_WARPS) {
        const int rl = x / chunks, ch = x % chunks, gr = j.row0 + 32 * blockIdx.y + rl;
        if (32 * (int)blockIdx.y + rl < j.rows)
            *reinterpret_cast<uint4 *>(a.y + (j.q0 + gr / a.group) * a.y_token +
                                       (j.head * (int)a.group.d + gr % a.group) * a.y_head + 8 * ch) =
                *reinterpret_cast<const uint4 *>(&out[rl][8 * ch]);
    }
}

// The register split needs what the compiler gave each thread at launch: a
// kernel launched with fewer would wait for registers that never come.
template <int DP>
bool regs_ok() {
    static const bool ok = [] {
        cudaFuncAttributes f;
        if (cudaFuncGetAttributes(&f, attn_tc_kernel<DP>) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        return f.numRegs == REGS_LAUNCH;
    }();
    return ok;
}

template <int DP>
int launch_tc(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    static_assert(TcCfg<DP>::SMEM + sizeof(PlanShared) <= 227 * 1024, "shared memory");
    if (!regs_ok<DP>()) return W4_ERR_DEVICE;
    if (!set_smem_once(reinterpret_cast<const void *>(attn_tc_kernel<DP>), (int)TcCfg<DP>::SMEM)) return W4_ERR_LAUNCH;
    attn_tc_kernel<DP><<<grid, TC_THREADS, TcCfg<DP>::SMEM, stream>>>(mk, mv, a);
    const int st = launch_status();
    return st != W4A16_OK ? st : launch_dependent(join_tc_kernel, dim3(grid, QROWS / 32), 32 * JOIN_WARPS, a, stream);
}

}  // namespace

int attn_tc_rows() { return QROWS; }

int attn_tc_launch(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    return a.head_dim <= 64 ? launch_tc<64>(mk, mv, a, grid, stream) : launch_tc<128>(mk, mv, a, grid, stream);
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
