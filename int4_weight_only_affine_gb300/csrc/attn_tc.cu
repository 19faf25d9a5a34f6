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
//  * Warp 8: copies K and V tiles page by page (tensor copies) into a ring.
//  * Warp 9: one thread issues S_t = Q_t K^T (both operands in shared memory)
//    and O_t += P_t V (P_t from tensor memory).
//  * Warps 0-3 and 4-7: softmax of tile 0 and 1, one thread to a row, so row
//    maxima and sums need no exchange.  O_t is rescaled in tensor memory only
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
constexpr int TC_THREADS = 320;
constexpr int HALF = KEYS * 128;  // bytes of 64 columns of 128 rows
constexpr float kGrow = 8.f;      // growth of the maximum (base 2) that rescales
constexpr float kLn2 = 0.69314718055994531f;

template <int DP>
struct TcCfg {
    static constexpr int HALVES = DP / 64;
    static constexpr int TILE = HALVES * HALF;                    // 128 rows of Q, K or V
    static constexpr int SLOTS = DP == 64 ? 8 : 5;                // ring of K and V tiles
    static constexpr int BARS = 2 * SLOTS + 2 * 4 + 1;
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
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
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
    auto p_full = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 4 + t); };  // P_t written (and S_t read, O_t rescaled)
    auto o_done = [&](int t) { return bar0 + 8u * (2 * C::SLOTS + 6 + t); };  // O_t += P_t V done
    const uint32_t end_bar = bar0 + 8u * (2 * C::SLOTS + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::SLOTS; ++s) {
            mbar_init(kv_full(s), 1);
            mbar_init(kv_empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full(t), 128);
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t), 128);
            mbar_init(o_done(t), 1);
        }
        mbar_init(end_bar, 1);
        *abort = 0;
        a.joins[blockIdx.x].parts = 0;
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

    if (warp == 8) {
        // ---------------- copies: K and V of every unit, in turn ----------------
        const int boxes = KEYS / a.box_rows * C::HALVES;
        int it = 0;
        bool ok = true;
        while (ok && pc.next()) {
            for (int i = 0; ok && i < 2 * pc.n; ++i) {
                const int st = it % C::SLOTS;
                ok = __all_sync(~0u, mbar_wait(kv_empty(st), ((it / C::SLOTS) & 1) ^ 1, abort));
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(kv_full(st), C::TILE);
                __syncwarp();
                const int p0 = (pc.it.t0 + pc.tile0 + (i >> 1)) * KEYS;
                for (int x = lane; x < boxes; x += 32) {
                    const int half = x % C::HALVES, row = x / C::HALVES * a.box_rows, p = p0 + row;
                    const int page = page_of(a, pc.b, p, pc.it.lo, pc.it.hi);
                    tma_load_4d(ring + st * C::TILE + half * HALF + row * 128, i & 1 ? &map_v : &map_k, 64 * half,
                                p % a.page_size, pc.head, page, kv_full(st));
                }
                ++it;
            }
        }
        // Every copy has landed before the CTA may exit.
        __syncwarp();
        if (lane == 0)
            for (int k = max(0, it - C::SLOTS); k < it; ++k) mbar_wait(kv_full(k % C::SLOTS), (k / C::SLOTS) & 1);
    } else if (warp == 9) {
        // ---------------- MMA issue ----------------
        if (lane == 0) {
            constexpr uint32_t id_s = instr_desc(KEYS, 0), id_o = instr_desc(DP, 1);
            int it = 0;             // ring position
            uint32_t nq = 0;        // pieces begun
            uint32_t steps[2] = {0, 0};  // P_t V products issued so far
            bool ok = true;
            auto wait_slot = [&](int k) {
                ok = ok && mbar_wait(kv_full(k % C::SLOTS), (k / C::SLOTS) & 1, abort);
                fence_after();
            };
            auto score = [&](int t, int k) {  // S_t = Q_t K^T
                const uint32_t q = base + t * C::TILE, kt = ring + k % C::SLOTS * C::TILE;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s) {
                    const uint32_t off = (s / 4) * HALF + (s % 4) * 32;
                    mma_ss(tmem + C::S0 + 128 * t, operand_desc(q + off, 16, 1024), operand_desc(kt + off, 16, 1024),
                           id_s, s != 0);
                }
                commit(s_full(t));
            };
            uint32_t begun[2] = {0, 0};  // pieces of tile t
            while (ok && pc.next()) {
                const int nt = pc.rows() > 128 ? 2 : 1;
                ++nq;
                for (int t = 0; t < nt; ++t) {
                    ok = ok && mbar_wait(q_full(t), begun[t] & 1, abort);
                    ++begun[t];
                    // the columns of S_t, if P_t lies there: the last product of the piece before has read it
                    if (C::P_IN_S && steps[t] > 0) ok = ok && mbar_wait(o_done(t), (steps[t] - 1) & 1, abort);
                    if (t == 0) wait_slot(it);
                    if (!ok) break;
                    fence_after();
                    score(t, it);
                }
                if (!ok) break;
                commit(kv_empty(it % C::SLOTS));
                for (int j = 0; ok && j < pc.n; ++j) {
                    const int kv = it + 1, kn = it + 2;
                    const bool more = j + 1 < pc.n;
                    for (int t = 0; t < nt; ++t) {
                        if (t == 0) wait_slot(kv);
                        ok = ok && mbar_wait(p_full(t), steps[t] & 1, abort);
                        if (!ok) break;
                        fence_after();
                        const uint32_t vt = ring + kv % C::SLOTS * C::TILE;
#pragma unroll
                        for (int s = 0; s < KEYS / 16; ++s)
                            mma_ts(tmem + C::O0 + DP * t, tmem + C::P0 + C::P_STEP * t + 8 * s,
                                   operand_desc(vt + s * 2048, HALF, 1024), id_o, (j | s) != 0);
                        commit(o_done(t));
                        if (t == nt - 1) commit(kv_empty(kv % C::SLOTS));
                        ++steps[t];
                        if (more) {
                            if (t == 0) wait_slot(kn);
                            if (C::P_IN_S) ok = ok && mbar_wait(o_done(t), (steps[t] - 1) & 1, abort);
                            if (!ok) break;
                            score(t, kn);
                            if (t == nt - 1) commit(kv_empty(kn % C::SLOTS));
                        }
                    }
                    it += 2;
                }
            }
            commit(end_bar);  // every product is done before the CTA may exit
            mbar_wait(end_bar, 0);
        }
        __syncwarp();
    } else {
        // ---------------- softmax: warps 4 t .. 4 t + 3 for tile t, one thread to a row ----------------
        const int t = warp >> 2, quad = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t s_at = lanes + C::S0 + 128 * t, p_at = lanes + C::P0 + C::P_STEP * t, o_at = lanes + C::O0 + DP * t;
        uint32_t steps = 0;
        int it = 0;
        while (pc.next()) {
            const int first_slot = it;
            it += 2 * pc.n;
            const int rows = pc.rows(), row0 = pc.row0();
            if (128 * t >= rows) continue;
            // Q_t: the warp's 32 rows, 16 bytes a lane, swizzled.
            for (int x = lane; x < 32 * (DP / 8); x += 32) {
                const int rl = 32 * quad + x / (DP / 8), ch = x % (DP / 8), r = 128 * t + rl, gr = row0 + r;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows && 8 * ch < a.head_dim)
                    v = *reinterpret_cast<const uint4 *>(a.q + (pc.s.q0 + gr / a.group) * a.q_token +
                                                         (pc.head * a.group + gr % a.group) * a.q_head + 8 * ch);
                const uint32_t at = base + t * C::TILE + (ch / 8) * HALF + rl * 128 + (((ch ^ rl) & 7) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                             : "memory");
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full(t));

            const int r = 128 * t + 32 * quad + lane;  // this thread's row of the item
            const bool in = r < rows;
            const int gr = row0 + r;
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
                mbar_wait(s_full(t), steps & 1, abort);
                fence_after();
                uint32_t sr[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load(s_at + 32 * c, sr[c]);
                tmem_load_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_loaded(sr[c]);
                if (j0 + KEYS > all_ub || j0 < all_lb) {
                    const int lo = lb - j0, hi = ub - j0;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i < lo || 32 * c + i >= hi) sr[c][i] = 0xFF800000u;  // -infinity
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], __uint_as_float(sr[c][i]));
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale;
                const bool grow = mx > ref + kGrow || (ref == -INFINITY && mx > ref);
                if (__any_sync(~0u, grow)) {
                    const float nr = grow ? mx : ref;
                    const float c = ref == -INFINITY ? 0.f : exp2_approx(ref - nr);
                    if (j > 0) {
                        mbar_wait(o_done(t), (steps - 1) & 1, abort);
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
                const float base2 = ref == -INFINITY ? 0.f : ref;
                float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pr[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float e0 = exp2_approx(fmaf(__uint_as_float(sr[2 * h + i / 16][2 * i % 32]), a.scale, -base2));
                        const float e1 = exp2_approx(fmaf(__uint_as_float(sr[2 * h + i / 16][2 * i % 32 + 1]), a.scale, -base2));
                        s4[i & 3] += e0 + e1;
                        pr[i] = pack2(e0, e1);
                    }
                    tmem_store(p_at + 32 * h, pr);
                }
                sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                if (t == 0 && (j0 < pc.it.lo || j0 + KEYS > pc.it.hi)) {
                    // Rows of V that the item does not see: one to a thread.
                    const int k = first_slot + 2 * j + 1, row = 32 * quad + lane;
                    mbar_wait(kv_full(k % C::SLOTS), (k / C::SLOTS) & 1, abort);
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
                tmem_store_wait();
                fence_before();
                mbar_arrive(p_full(t));
            }

            // ---------------- the piece's rows ----------------
            mbar_wait(o_done(t), (steps - 1) & 1, abort);
            fence_after();
            const bool whole = pc.begins && pc.ends;
            const long long tok = pc.s.q0 + gr / a.group;
            const int head = pc.head * a.group + gr % a.group;
            const long long prow = (long long)pc.slot() * QROWS + r;
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            if (in) {
                if (!whole)
                    reinterpret_cast<float2 *>(a.part_ml)[prow] = make_float2(ref, sum);
                else if (a.lse)
                    a.lse[tok * (a.kv_heads * a.group) + head] = sum > 0.f ? (ref + log2f(sum)) * kLn2 : -INFINITY;
            }
            if (threadIdx.x == 0 && pc.begins && !pc.ends)
                a.joins[blockIdx.x] = JoinItem{pc.parts(plan), pc.s.q0, pc.head, row0, rows};
#pragma unroll 1
            for (int cb = 0; cb < DP / 32; ++cb) {
                uint32_t o[32];
                tmem_load(o_at + 32 * cb, o);
                tmem_load_wait();
                tmem_loaded(o);
                if (!in) continue;
                if (whole) {
                    uint16_t *dst = a.y + tok * a.y_token + head * a.y_head + 32 * cb;
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (32 * cb + i < a.head_dim) {
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                h[e] = pack2(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                } else {
                    float *dst = a.part_o + prow * a.head_dim + 32 * cb;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (32 * cb + i < a.head_dim)
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
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

template <int DP>
int launch_tc(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    static_assert(TcCfg<DP>::SMEM + sizeof(PlanShared) <= 227 * 1024, "shared memory");
    if (!set_smem_once(reinterpret_cast<const void *>(attn_tc_kernel<DP>), (int)TcCfg<DP>::SMEM)) return W4_ERR_LAUNCH;
    attn_tc_kernel<DP><<<grid, TC_THREADS, TcCfg<DP>::SMEM, stream>>>(mk, mv, a);
    return launch_status();
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
