// f16_attention for few query rows (decode steps, drafted tokens, short
// chunks), the join of split items, and the call's entry points.
//
// y = sum_j softmax_j(scale q k_j) v_j in one pass over the positions: with
// the scores in powers of two, s_j = scale log2(e) q k_j, a running maximum m
// and running sums l = sum 2^(s_j - m), o = sum 2^(s_j - m) v_j are corrected
// by 2^(m_old - m_new) whenever m grows; partial (m, l, o) of disjoint
// positions combine the same way.
//
// With few rows per key the pass is bound by reading K and V once: 4
// head_dim bytes a position.  One persistent CTA per SM works through its
// range of units (attn.cuh).  A producer warp copies the tiles, K and V of
// KEYS positions each, page by page, with tensor copies into a ring of up to
// 192 KB.  The other warps each own 16 positions of every tile, and keep
// their own (m, l, o) of 16 rows in registers for the whole item: no warp
// waits for another inside the loop.  16 x 16 scores and their product with V
// are m16n8k16 tensor-core products, far below their rate here; the warps'
// sums are merged through shared memory at the end of the item.
//
// Measured (heads of 128, pages of 16 to 64): single tokens of 48 sequences of
// up to 8192 positions, 8 key/value heads, 534 MB, 100 us, 5.3 TB/s (80% of a plain copy's
// rate; while all SMs stream, 6.2); one of 131071 positions, 134 MB, 34 us, 3.9
// TB/s: the start (5000 cycles until the first tile is there) and the join of
// 76 parts (10000) are a third of it.  One short sequence, 600 positions,
// takes 9.6 us, a chain of latencies: plan 2500 cycles, page look-up and first
// copy 3700, one tile 1700, the warps' merge 2000, counting the part in and
// waiting for the others 3000, join 2000.
#include <math.h>
#include <string.h>

#include <type_traits>

#include "attn.cuh"

namespace w4a16 {

// attn_tc.cu
int attn_tc_launch(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream);
int attn_tc_rows();
int attn_tc_status();

namespace {

constexpr int kMaxGrid = 256;  // CTAs of a launch, >= the SMs of the GPU
constexpr float kLog2e = 1.4426950408889634f;

template <int DP>
struct RowCfg {
    static constexpr int ROWS = 16;
    static constexpr int KEYS = kv_tile(DP);
    using Work = Cut<ROWS, KEYS, 2, 1, ROWS, 4, 1, false>;
    static constexpr int WARPS = KEYS / 16;             // consumers
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int TILE = KEYS * 128 * (DP / 64); // bytes of K or V
    static constexpr int STAGES = 192 * 1024 / (2 * TILE);
    static constexpr int MERGE = WARPS * ROWS * 36 * 4; // 32 columns of every warp's rows, or 64 of 8 rows, and padding
    static constexpr int ML = (WARPS + 1) * ROWS * 8;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * 2 * TILE + MERGE + ML + 16 * STAGES + 16;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
// Joins rows of a shared item, by WARPS warps.  A part's rows lie one after the
// other; lane l takes the columns 4 l .. 4 l + 3, and those 128 further on.
template <int DP, int WARPS, int ROWS>
struct Join {
    static constexpr int H = DP > 128 ? 2 : 1, FLIGHT = 10 / H;  // parts of a row whose loads are in flight
    const AttnArgs &a;
    const Part &part;

    // Sums of row r over the parts i0, i0 + STEP, ...
    template <int STEP>
    __device__ __forceinline__ void sum_parts(int r, int i0, float &mx, float &sum, float4 (&acc)[2]) const {
        const int lane = threadIdx.x & 31;
        const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
        mx = -INFINITY;
        sum = 0.f;
        acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (; i0 < part.parts; i0 += FLIGHT * STEP) {
            float4 v[FLIGHT][H];
            float2 c[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const int i = i0 + k * STEP;
                c[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int h = 0; h < H; ++h) v[k][h] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < part.parts) {
                    const long long row = part_slot(part.first, i) * ROWS + r;
                    c[k] = __ldcg(ml + row);
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        if (128 * h + 4 * lane < a.head_dim)
                            v[k][h] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + row * a.head_dim + 128 * h + 4 * lane));
                }
            }
            float top = mx;
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) top = fmaxf(top, c[k].x);
            const float f0 = corr(mx, top);
            mx = top;
            sum *= f0;
#pragma unroll
            for (int h = 0; h < H; ++h) scale4(acc[h], f0);
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                const float f = corr(c[k].x, top);
                sum += c[k].y * f;
#pragma unroll
                for (int h = 0; h < H; ++h) add4(acc[h], v[k][h], f);
            }
        }
    }
    __device__ __forceinline__ static void scale4(float4 &o, float f) {
        o.x *= f;
        o.y *= f;
        o.z *= f;
        o.w *= f;
    }
    __device__ __forceinline__ static void add4(float4 &o, const float4 &v, float f) {
        o.x += v.x * f;
        o.y += v.y * f;
        o.z += v.z * f;
        o.w += v.w * f;
    }
    // Columns 128 h + 4 lane .. of row r.
    __device__ __forceinline__ void write(int r, int h, float mx, float sum, const float4 &o) const {
        const int lane = threadIdx.x & 31, c = 128 * h + 4 * lane;
        if (c >= a.head_dim) return;
        const int gr = part.row0 + r, head = part.head * (int)a.group.d + gr % a.group;
        const long long tok = part.q0 + gr / a.group;
        const float inv = inverse(sum);
        *reinterpret_cast<uint2 *>(a.y + tok * a.y_token + head * a.y_head + c) =
            make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
        if (a.lse && c == 0) a.lse[tok * (a.kv_heads * (int)a.group.d) + head] = log_sum(mx, sum);
    }

    // Rows r0, r0 + step, ..  Of few parts: a warp to a row, all its parts in
    // flight at once.  Of many: all warps to a row, which take the parts in
    // turn and merge through sh.
    template <class Sync>
    __device__ __forceinline__ void rows(int r0, int step, float *sh, Sync sync) const {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float mx, sum;
        float4 acc[2];
        if (part.parts <= FLIGHT) {
#pragma unroll 1
            for (int r = r0 + warp * step; r < part.rows; r += WARPS * step) {
                sum_parts<1>(r, 0, mx, sum, acc);
#pragma unroll
                for (int h = 0; h < H; ++h) write(r, h, mx, sum, acc[h]);
            }
            return;
        }
        float4 *sh_o = reinterpret_cast<float4 *>(sh);                        // [WARPS][2][32]
        float2 *sh_ml = reinterpret_cast<float2 *>(sh + WARPS * 2 * 32 * 4);  // [WARPS]
#pragma unroll 1
        for (int r = r0; r < part.rows; r += step) {
            sum_parts<WARPS>(r, warp, mx, sum, acc);
#pragma unroll
            for (int h = 0; h < H; ++h) sh_o[(warp * 2 + h) * 32 + lane] = acc[h];
            if (lane == 0) sh_ml[warp] = make_float2(mx, sum);
            sync();
            if (warp < H) {
                mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, sh_ml[w].x);
                sum = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float f = corr(sh_ml[w].x, mx);
                    sum += sh_ml[w].y * f;
                    add4(o, sh_o[(w * 2 + warp) * 32 + lane], f);
                }
                write(r, warp, mx, sum, o);
            }
            sync();
        }
    }
};

// WIDE: the tensor maps copy whole heads.
template <int DP, bool WIDE>
__global__ void __launch_bounds__(RowCfg<DP>::THREADS, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ AttnArgs a) {
    using C = RowCfg<DP>;
    constexpr int ROWS = C::ROWS, KEYS = C::KEYS, NT = 32 * C::WARPS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PlanShared plan_sh;
    const uint32_t raw = (uint32_t)__cvta_generic_to_shared(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    float *merge = reinterpret_cast<float *>(gbase + C::STAGES * 2 * C::TILE);
    float2 *ml_sh = reinterpret_cast<float2 *>(gbase + C::STAGES * 2 * C::TILE + C::MERGE);
    float2 *row_sh = ml_sh + C::WARPS * ROWS;
    const uint32_t bar0 = base + C::STAGES * 2 * C::TILE + C::MERGE + C::ML;
    volatile int *abort = reinterpret_cast<volatile int *>(gbase + (bar0 - base) + 16 * C::STAGES);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), C::WARPS);
        }
        *abort = 0;
        prefetch_maps(&map_k, &map_v);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    make_plan<typename C::Work, C::THREADS>(a, plan_sh);  // (its barriers also publish the above)
    const Plan plan = plan_sh.plan;
    Pieces<typename C::Work> pc(a, plan);

    if (warp == C::WARPS) {
        // ---------------- producer ----------------
        constexpr int HALVES = DP / 64;
        const int boxes = KEYS / a.box_rows;  // at most 16
        int it = 0;
        bool ok = true;
        while (ok && uniform(pc.next())) {
            const int n = uniform(pc.n), head = uniform(pc.head);
            int p0 = uniform(pc.it.t0 + pc.tile0) * KEYS;
            for (int i = 0; i < n; ++i, ++it, p0 += KEYS) {
                const int st = it % C::STAGES;
                const int page = lane < boxes ? page_of(a, pc.b, p0 + lane * a.box_rows, pc.it.lo, pc.it.hi) : 0;
                ok = __all_sync(~0u, wait(empty_bar(st), ((it / C::STAGES) & 1) ^ 1, abort));
                if (!ok) break;
                const uint32_t kdst = base + st * 2 * C::TILE, vdst = kdst + C::TILE, bar = full_bar(st);
                if (elect_one()) mbar_expect_tx(bar, 2 * C::TILE);
                for (int x = 0; x < boxes; ++x) {
                    const int pg = __shfl_sync(~0u, page, x), row = x * a.box_rows, at = (p0 + row) % a.page_size;
                    if (!elect_one()) continue;
                    if (WIDE) {
                        tma_load_5d(kdst + row * HALVES * 128, &map_k, 0, at, 0, head, pg, bar);
                        tma_load_5d(vdst + row * HALVES * 128, &map_v, 0, at, 0, head, pg, bar);
                    } else {
#pragma unroll
                        for (int half = 0; half < HALVES; ++half) {
                            const uint32_t off = row * HALVES * 128 + half * a.box_rows * 128;
                            tma_load_4d(kdst + off, &map_k, 64 * half, at, head, pg, bar);
                            tma_load_4d(vdst + off, &map_v, 64 * half, at, head, pg, bar);
                        }
                    }
                }
            }
        }
        // Every copy has landed before the CTA may exit.
        for (int k = max(0, it - C::STAGES); k < it; ++k) wait(full_bar(k % C::STAGES), (k / C::STAGES) & 1, nullptr);
        return;
    }

    // ---------------- consumers ----------------
    // A tile lies copy by copy, each as columns of 64 of its box_rows rows.
    // 8-row groups start on 1024 bytes, so a row's swizzle is that of row % 8.
    const uint32_t half_bytes = a.box_rows * 128;
    auto row_at = [&](int row) {
        const int box = row & ~(a.box_rows - 1);
        return (uint32_t)(box * (DP / 64) * 128 + (row - box) * 128);
    };
    // Lane l addresses row (l & 7) + 8 (l >> 4) of its warp's 16 positions of K, 8-column chunk (l >> 3) & 1: registers
    // 0, 1 of a load are the two chunks of positions 0-7, registers 2, 3 of positions 8-15.
    const int krow = (lane & 7) + 8 * (lane >> 4), kch = (lane >> 3) & 1;
    const uint32_t k_off = row_at(16 * warp + krow);
    // And position l & 15, 8-column chunk l >> 4 of V.
    const int vrow = lane & 15, vch = lane >> 4;
    const uint32_t v_off = row_at(16 * warp + vrow);
    const int g = lane >> 2, t4 = lane & 3;
    if (threadIdx.x == NT - 32) {  // (off the way: the first positions are being copied)
        const Begin begin = cta_begins(a);
        plan_sh.begun_before = begin.before;
        cta_has_begun(a, begin);
    }
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory"); };
    Part shared0, shared1;  // items that this CTA shares with earlier and later ones
    unsigned seen0 = 0, seen1 = 0;  // (thread 0) their counts with this CTA's part
    bool waits = true;              // and whether it may wait for the others'
    int shares = 0;
    int it = 0;
    while (pc.next()) {
        const int row0 = pc.row0(), rows = pc.rows();
        // Query fragments, and the positions each of this lane's rows sees.
        uint32_t qf[DP / 16][4];
        int lb[2], ub[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int r = row0 + 8 * hf + g;
            const bool in = r < row0 + rows;
            const int tok = r / a.group, p = pc.s.kv - pc.s.qn + tok;
            ub[hf] = in ? (a.causal ? min(p + 1, pc.s.kv) : pc.s.kv) : 0;
            lb[hf] = a.window > 0 ? p - a.window + 1 : 0;
            const uint16_t *qr = a.q + (pc.s.q0 + tok) * a.q_token +
                                 (pc.head * (int)a.group.d + r % a.group) * a.q_head;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                const int c = 16 * k + 2 * t4;
                qf[k][hf] = in && c < a.head_dim ? *reinterpret_cast<const uint32_t *>(qr + c) : 0u;
                qf[k][2 + hf] =
                    in && c + 8 < a.head_dim ? *reinterpret_cast<const uint32_t *>(qr + c + 8) : 0u;
            }
        }
        // Tiles inside these bounds need no mask for any row of the item.
        const int pf = pc.s.kv - pc.s.qn + row0 / a.group, pl = pc.s.kv - pc.s.qn + (row0 + rows - 1) / a.group;
        const int all_ub = a.causal ? min(pf + 1, pc.s.kv) : pc.s.kv;
        const int all_lb = a.window > 0 ? pl - a.window + 1 : 0;

        float o[DP / 8][4], m[2], l[2];
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

        for (int i = 0; i < pc.n; ++i, ++it) {
            const int st = it % C::STAGES;
            const int j0 = (pc.it.t0 + pc.tile0 + i) * KEYS + 16 * warp;  // this warp's first position
            const uint32_t kb = base + st * 2 * C::TILE, vb = kb + C::TILE;
            wait(full_bar(st), (it / C::STAGES) & 1, abort);
            const bool outside = j0 < pc.it.lo || j0 + 16 > pc.it.hi;
            if (outside) {
                // Rows of V that the item does not see hold anything; 0 x NaN must not reach the sums.
                for (int x = lane; x < 16 * (DP / 8); x += 32) {
                    const int row = x / (DP / 8), ch = x % (DP / 8);
                    if (j0 + row < pc.it.lo || j0 + row >= pc.it.hi) {
                        const uint32_t at = vb + row_at(16 * warp + row) + (ch / 8) * half_bytes + (((ch ^ row) & 7) << 4);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    }
                }
                __syncwarp();
            }
            if (j0 < pc.it.hi && j0 + 16 > pc.it.lo) {
                // Two sums of half the columns each: shorter chains of dependent products.
                float s[2][4], s2[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    uint32_t kf[4];
                    const int ch = 2 * k + kch;
                    ldsm4(kf, kb + k_off + (ch / 8) * half_bytes + (((ch ^ krow) & 7) << 4));
                    auto &d = k & 1 ? s2 : s;
                    mma_16816(d[0], qf[k][0], qf[k][1], qf[k][2], qf[k][3], kf[0], kf[1]);
                    mma_16816(d[1], qf[k][0], qf[k][1], qf[k][2], qf[k][3], kf[2], kf[3]);
                }
                const bool masked = j0 + 16 > all_ub || j0 < all_lb;
                uint32_t pf4[4];
                float mx[2];
                bool grown = false;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                    const int j = j0 + 8 * n + 2 * t4 + (e & 1), hf = e >> 1;
                    s[n][e] = (s[n][e] + s2[n][e]) * a.scale;
                    if (masked && (j >= ub[hf] || j < lb[hf])) s[n][e] = -INFINITY;
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    mx[hf] = fmaxf(fmaxf(s[0][2 * hf], s[0][2 * hf + 1]),
                                       fmaxf(s[1][2 * hf], s[1][2 * hf + 1]));
#pragma unroll
                for (int step = 1; step <= 2; step <<= 1)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(~0u, mx[hf], step));
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) grown |= mx[hf] > m[hf];
                if (__any_sync(~0u, grown)) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float top = fmaxf(mx[hf], m[hf]), c = corr(m[hf], top);
                        m[hf] = top;
                        l[hf] *= c;
#pragma unroll
                        for (int n = 0; n < DP / 8; ++n) {
                            o[n][2 * hf] *= c;
                            o[n][2 * hf + 1] *= c;
                        }
                    }
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float ref = m[hf] == -INFINITY ? 0.f : m[hf];
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = exp2_approx(s[e >> 1][2 * hf + (e & 1)] - ref);
                    l[hf] += (p[0] + p[1]) + (p[2] + p[3]);
                    // Probabilities, at most 1, to binary16 for the product with V (the sum l keeps fp32).
                    pf4[hf] = pack2(p[0], p[1]);
                    pf4[2 + hf] = pack2(p[2], p[3]);
                }
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    uint32_t vf[4];
                    const int ch = 2 * n + vch;
                    ldsm4t(vf, vb + v_off + (ch / 8) * half_bytes + (((ch ^ vrow) & 7) << 4));
                    mma_16816(o[2 * n], pf4[0], pf4[1], pf4[2], pf4[3], vf[0], vf[1]);
                    mma_16816(o[2 * n + 1], pf4[0], pf4[1], pf4[2], pf4[3], vf[2], vf[3]);
                }
            }
            if (outside) fence_proxy_async_smem();  // the zeros above, before the next copy into the slot
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(st));
        }

        // ---------------- merge the warps' sums ----------------
        const bool whole = pc.begins && pc.ends;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float v = l[hf];
            v += __shfl_xor_sync(~0u, v, 1);
            v += __shfl_xor_sync(~0u, v, 2);
            if (t4 == 0) ml_sh[warp * ROWS + 8 * hf + g] = make_float2(m[hf], v);
        }
        sync();
        if ((int)threadIdx.x < rows) {  // a row's maximum and sum over the warps; what its outputs are scaled by
            const int r = threadIdx.x;
            float2 w[C::WARPS];
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < C::WARPS; ++i) {
                w[i] = ml_sh[i * ROWS + r];
                mx = fmaxf(mx, w[i].x);
            }
#pragma unroll
            for (int i = 0; i < C::WARPS; ++i) sum += w[i].y * corr(w[i].x, mx);
            row_sh[r] = make_float2(mx, whole ? inverse(sum) : 1.f);
            if (!whole) {
                reinterpret_cast<float2 *>(a.part_ml)[(long long)pc.slot() * ROWS + r] = make_float2(mx, sum);
            } else if (a.lse) {
                const int gr = row0 + r;
                a.lse[(long long)(pc.s.q0 + gr / a.group) * (a.kv_heads * (int)a.group.d) + pc.head * (int)a.group.d +
                      gr % a.group] = log_sum(mx, sum);
            }
        }
        sync();
        float f[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const float2 w = row_sh[8 * hf + g];
            f[hf] = corr(m[hf], w.x) * w.y;
        }
        // Outputs, COLS columns of HALVES x 8 rows at a time.
        auto merge_rows = [&](auto halves) {
            constexpr int HALVES = decltype(halves)::value, COLS = HALVES == 1 ? 64 : 32, LD = COLS + 8 / HALVES;
#pragma unroll
            for (int cb = 0; cb < DP / COLS; ++cb) {
#pragma unroll
                for (int n = 0; n < COLS / 8; ++n)
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                    *reinterpret_cast<float2 *>(&merge[(warp * 8 * HALVES + 8 * h + g) * LD + 8 * n + 2 * t4]) =
                        make_float2(o[COLS / 8 * cb + n][2 * h] * f[h], o[COLS / 8 * cb + n][2 * h + 1] * f[h]);
                sync();
                for (int x = threadIdx.x; x < 8 * HALVES * (COLS / 4); x += NT) {
                    const int r = x / (COLS / 4), c = 4 * (x % (COLS / 4)), col = COLS * cb + c;
                    if (r >= rows || col >= a.head_dim) continue;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < C::WARPS; ++w) {
                        const float4 u = *reinterpret_cast<const float4 *>(&merge[(w * 8 * HALVES + r) * LD + c]);
                        v.x += u.x;
                        v.y += u.y;
                        v.z += u.z;
                        v.w += u.w;
                    }
                    if (whole) {
                        const int gr = row0 + r;
                        uint16_t *dst = a.y + (pc.s.q0 + gr / a.group) * a.y_token +
                                        (pc.head * (int)a.group.d + gr % a.group) * a.y_head + col;
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
                    } else {
                        *reinterpret_cast<float4 *>(a.part_o + ((long long)pc.slot() * ROWS + r) * a.head_dim + col) = v;
                    }
                }
                sync();
            }
        };
        if (rows <= 8)
            merge_rows(std::integral_constant<int, 1>());
        else
            merge_rows(std::integral_constant<int, 2>());
        if (!whole) {
            const Part part = pc.part(plan);
            const unsigned count = threadIdx.x == 0 ? count_part<false>(a, part, plan_sh.begun_before, waits) : 0;
            if (shares++ == 0) {
                shared0 = part;
                seen0 = count;
            } else {
                shared1 = part;
                seen1 = count;
            }
        }
    }

    // ---------------- join this CTA's rows of the items it shares ----------------
    for (int i = 0; i < shares; ++i) {
        const Part part = i == 0 ? shared0 : shared1;
        const int joiners = min(part.parts, part.rows);
        if (threadIdx.x == 0) {
            const unsigned seen = i == 0 ? seen0 : seen1;
            // (A CTA with no share of the rows need not wait.  One that said it would not may be the last to count.)
            *abort = await_parts(a, part, seen, part.index < joiners && waits, part.parts);
        }
        sync();
        const int mode = *abort;
        const Join<DP, C::WARPS, ROWS> join{a, part};
        const bool all = mode == kJoinAll;
        if (all || (mode == kJoinShare && part.index < joiners))
            join.rows(all ? 0 : part.index, all ? 1 : joiners, merge, sync);
        sync();
        if (threadIdx.x == 0) part_done(a, part);
    }
}

template <int DP, bool WIDE>
int launch_rows(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    using C = RowCfg<DP>;
    static_assert(C::SMEM + sizeof(PlanShared) <= 227 * 1024, "shared memory");
    if (!ensure_smem(reinterpret_cast<const void *>(attn_rows_kernel<DP, WIDE>), C::SMEM)) return W4_ERR_LAUNCH;
    return launch_dependent(attn_rows_kernel<DP, WIDE>, grid, C::THREADS, C::SMEM, stream, mk, mv, a);
}

// Whether a call takes the tcgen05 kernel: more rows per sequence and
// key/value head than one tile of the row kernel, heads of at most 128 (wider
// ones leave no room for two tiles' scores and sums in tensor memory).  With
// 16 rows the row kernel is faster at most sizes (16 sequences of 300
// positions, 8 heads of 128: 9.8 us against 13.4; 48 of 2720: 105 against 109;
// one of 16384: 20.5 against 22; but four of 16384: 64 against 56); above, it
// reads every key and value once per 16 rows (20 rows, the same sizes: 32, 188
// and 27 against 22, 108 and 21).
bool takes_tc(int group, int head_dim, int max_q_len) { return (long long)group * max_q_len > 16 && head_dim <= 128; }

// Workspace: the counters, then two partial tiles per CTA (statistics, outputs).
constexpr size_t kCounterBytes = (2 * kMaxGrid + 4) * sizeof(unsigned);
size_t workspace_need(int rows, int head_dim) {
    return (kCounterBytes + (size_t)2 * kMaxGrid * rows * (2 + head_dim) * 4 + 15) / 16 * 16;
}

}  // namespace

// Reads and clears this translation unit's records: bit 0 an expired wait, bit 1 a bad index; -1 on error.
int attn_status() {
    int w = 0, b = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&w, g_wait_expired, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&b, g_bad_index, sizeof(int)) != cudaSuccess)
        return -1;
    const int tc = attn_tc_status();
    if (tc < 0) return -1;
    if (w) cudaMemcpyToSymbol(g_wait_expired, &zero, sizeof(int));
    if (b) cudaMemcpyToSymbol(g_bad_index, &zero, sizeof(int));
    return (w ? 1 : 0) | (b ? 2 : 0) | tc;
}
}  // namespace w4a16

using namespace w4a16;

extern "C" size_t f16_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q_len) {
    if (kv_heads < 1 || kv_heads > kMaxHeads || q_heads < kv_heads || q_heads % kv_heads != 0 ||
        q_heads / kv_heads > kMaxHeads || !head_dim_ok(head_dim) || max_q_len < 0)
        return 0;
    return workspace_need(takes_tc(q_heads / kv_heads, head_dim, max_q_len) ? attn_tc_rows() : 16, head_dim);
}

extern "C" int f16_attention(const uint16_t *q, int64_t q_token, int64_t q_head, uint16_t *y, int64_t y_token,
                             int64_t y_head, float *lse, int q_heads, float scale, int causal, int window,
                             const f16_kv_cache *cache, const f16_kv_batch *batch, void *workspace,
                             size_t workspace_bytes, void *stream) {
    int st = check_cache(cache);
    if (st != W4A16_OK) return st;
    AttnArgs a;
    st = check_batch(batch, cache->page_size, a.b);
    if (st != W4A16_OK) return st;
    const int heads = cache->heads, d = cache->head_dim;
    if (q_heads < heads || q_heads % heads != 0 || q_heads / heads > kMaxHeads || !(scale > 0.f) ||
        !(scale < INFINITY) || (causal & ~1) != 0 || window < 0 ||
        (long long)batch->total_q * (q_heads / heads) > 0x40000000ll)
        return W4_ERR_SHAPE;
    if (batch->total_q == 0) return W4A16_OK;
    if (!q || !y) return W4_ERR_NULL;
    if (!aligned16(q) || !aligned16(y) || !aligned16(workspace) || !stride_ok(q_token) || !stride_ok(q_head) ||
        !stride_ok(y_token) || !stride_ok(y_head) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return W4_ERR_ALIGN;
    if (!workspace || workspace_bytes < f16_attention_workspace_bytes(q_heads, heads, d, batch->max_q_len))
        return W4_ERR_WORKSPACE;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    const bool tc = takes_tc(q_heads / heads, d, batch->max_q_len);
    const int rows = tc ? attn_tc_rows() : 16;
    a.q = q;
    a.y = y;
    a.lse = lse;
    a.q_token = q_token;
    a.q_head = q_head;
    a.y_token = y_token;
    a.y_head = y_head;
    a.group = fast_div(q_heads / heads);
    a.kv_heads = heads;
    a.head_dim = d;
    a.causal = causal;
    a.window = window < 0x40000000 ? window : 0x40000000;
    a.num_pages = cache->num_pages;
    a.page_size = fast_div(cache->page_size);
    a.box_rows = cache->box_rows;
    a.few_tiles = (long long)batch->max_q_len * (q_heads / heads) <= 4 * rows;
    a.scale = scale * kLog2e;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    a.arrived = reinterpret_cast<unsigned *>(ws);
    a.left = a.arrived + kMaxGrid;
    a.begun = a.left + kMaxGrid;
    a.begun_before = a.begun + 1;
    a.taken = a.begun + 2;
    a.finished = a.begun + 3;
    a.part_ml = reinterpret_cast<float *>(ws + kCounterBytes);
    a.part_o = a.part_ml + (size_t)2 * kMaxGrid * rows * 2;
    const bool wide = !tc && d % 64 == 0 && d > 64;
    alignas(64) CUtensorMap mk, mv;
    memcpy(&mk, wide ? cache->k_wide : cache->k_map, sizeof(mk));
    memcpy(&mv, wide ? cache->v_wide : cache->v_map, sizeof(mv));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // No more CTAs than there can be units (lengths are known on the device only).
    const int keys = kv_tile(d);
    const long long tiles = ((long long)batch->total_q * (q_heads / heads) + rows - 1) / rows + batch->batch;
    const long long units = tiles * heads * (2ll * ((a.b.max_kv + keys - 1) / keys) + 8);  // (at their cost)
    if (units >= 0x7FFFFFFFll) return W4_ERR_SHAPE;
    int grid = sm_count() < kMaxGrid ? sm_count() : kMaxGrid;
    if (units < grid) grid = (int)units;
    a.may_queue = !a.few_tiles && tiles * heads > grid;
    if (tc) return attn_tc_launch(mk, mv, a, grid, s);
    if (d <= 64) return launch_rows<64, false>(mk, mv, a, grid, s);
    if (d == 128) return launch_rows<128, true>(mk, mv, a, grid, s);
    if (d < 128) return launch_rows<128, false>(mk, mv, a, grid, s);
    if (d == 192) return launch_rows<192, true>(mk, mv, a, grid, s);
    if (d < 192) return launch_rows<192, false>(mk, mv, a, grid, s);
    if (d == 256) return launch_rows<256, true>(mk, mv, a, grid, s);
    return launch_rows<256, false>(mk, mv, a, grid, s);
}
