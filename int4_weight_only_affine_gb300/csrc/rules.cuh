// Rules of token selection (w4_logit_rules): penalties of tokens that a request
// has seen, biases of listed tokens, and a mask, applied to the fp32 logits of a
// block's rows while they lie in shared memory, before the block selects from
// them.
//
// For logit l of token n in row m, with c = counts[slot[m]][n]:
//     c != 0:            z = l > 0 ? l / repetition : l * repetition
//     t = c & 0x7FFF:    z = z - frequency * t;   t != 0: z = z - presence
//     biases:            z = z + (sum of the row's values for n)
//     mask bit 0:        n cannot be selected
// each step one fp32 operation, rounded to nearest.  The rules read 2 bytes of
// counts and a bit of mask per logit, against the 0.5625 K bytes of weight that
// made it: they are bound by the latency of these reads, which a block therefore
// asks into L2 while it still streams weights.  Measured (bench of 16 rows of
// 151936, K = 2048, best 50, 300 biases a row): see lm_head_argmax_topk_rules.
#pragma once

#include "common.cuh"

namespace w4a16 {

struct Rules {
    const uint16_t *counts;  // null: no penalties
    long long stride;
    const int32_t *slot;
    const float *rep, *pres, *freq;  // null: 1, 0, 0
    const int32_t *boff, *btok;      // null: no biases
    const float *bval;
    const uint8_t *allowed;  // null: no mask
    long long astride;       // bytes from row to row
    int slots, entries;
    int vec;  // rows of counts start on 16 bytes
    int on;
};

// What stands in place of a masked logit: a NaN that no operation makes.
constexpr uint32_t kExcluded = 0xFFFFFFFFu;

// The slot of row m, or -1: no penalties (one out of range is reported).
__device__ __forceinline__ int rules_slot(const Rules &r, int m) {
    const int s = __ldg(r.slot + m);
    if (s >= r.slots) atomicExch(&g_bad_index, 1);
    return s < r.slots ? s : -1;
}

// Asks the counts and masks of tokens n0 .. n0 + rows - 1 into L2.
__device__ __noinline__ void rules_prefetch(const Rules &r, int M, int n0, int rows, int tid, int threads) {
    const int lines = (rows + 63) / 64;  // of 128 bytes: 64 counts, 1024 mask bits
    for (int e = tid; e < lines * M; e += threads) {
        const int m = e % M, n = n0 + e / M * 64;
        if (r.counts) {
            const int s = __ldg(r.slot + m);
            if (s >= 0 && s < r.slots) asm volatile("prefetch.global.L2 [%0];" ::"l"(r.counts + s * r.stride + n));
        }
        if (r.allowed && e / M % 16 == 0)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(r.allowed + m * r.astride + n / 8));
    }
}

// The logits res[i * M + m] of tokens n0 + i, i < rows (n0 a multiple of 16),
// under the rules.  Called by every thread of the block; a barrier before and after.
__device__ __noinline__ void rules_apply(const Rules &r, float *res, int M, int N, int n0, int rows, int tid,
                                         int threads) {
    // Eight tokens of one row of logits a thread: 16 bytes of counts, a byte of mask.
    for (int e = tid; e < (rows + 7) / 8 * M; e += threads) {
        const int m = e % M, i0 = e / M * 8;
        const int left = min(8, rows - i0);
        uint32_t bits = 0xFFu;
        if (r.allowed) bits = __ldg(r.allowed + m * r.astride + (n0 + i0) / 8);
        const int s = r.counts ? rules_slot(r, m) : -1;
        uint16_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        float rep = 1.f, pres = 0.f, freq = 0.f;
        if (s >= 0) {
            const uint16_t *src = r.counts + s * r.stride + n0 + i0;
            if (r.vec && left == 8) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < left) c[j] = __ldg(src + j);
            }
            if (r.rep) rep = __ldg(r.rep + m);
            if (r.pres) pres = __ldg(r.pres + m);
            if (r.freq) freq = __ldg(r.freq + m);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= left) break;
            float *p = res + (i0 + j) * M + m;
            if (!(bits >> j & 1u)) {
                *p = __uint_as_float(kExcluded);
            } else if (c[j]) {
                float z = *p;
                z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                const int t = c[j] & 0x7FFF;
                if (t) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)t)), pres);
                *p = z;
            }
        }
    }
    __syncthreads();
    if (!r.boff) return;
    // A warp takes a row's list, 32 entries at a time in order; entries of one
    // token inside a chunk are added up by the first of their lanes, in order.
    const int warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
    for (int m = warp; m < M; m += warps) {
        const int o0 = __ldg(r.boff + m), o1 = __ldg(r.boff + m + 1);
        if (o0 < 0 || o1 < o0 || o1 > r.entries) {
            if (lane == 0) atomicExch(&g_bad_index, 1);
            continue;
        }
        for (int at = o0; at < o1; at += 128) {
            int tok[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) tok[q] = at + 32 * q + lane < o1 ? __ldg(r.btok + at + 32 * q + lane) : -1;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (tok[q] >= N) atomicExch(&g_bad_index, 1);
                const bool mine = tok[q] >= n0 && tok[q] < n0 + rows;
                if (!__any_sync(~0u, mine)) continue;
                const float v = mine ? __ldg(r.bval + at + 32 * q + lane) : 0.f;
                const unsigned same = __match_any_sync(~0u, mine ? tok[q] : -1 - lane);
                float sum = v;
                if (__any_sync(~0u, mine && (same & (same - 1u)) != 0u)) {
                    sum = 0.f;
                    for (int l = 0; l < 32; ++l) {
                        const float w = __shfl_sync(~0u, v, l);
                        if (same >> l & 1u) sum = same & ((1u << l) - 1u) ? __fadd_rn(sum, w) : w;
                    }
                }
                if (mine && (same & ((1u << lane) - 1u)) == 0u) {
                    float *p = res + (tok[q] - n0) * M + m;
                    if (__float_as_uint(*p) != kExcluded) *p = __fadd_rn(*p, sum);
                }
                __syncwarp();
            }
        }
    }
    __syncthreads();
}

// Host checks of the rules for M rows of N logits; fills the device form.
inline int check_rules(const w4_logit_rules *u, int N, Rules &r) {
    r = Rules{};
    if (!u) return W4A16_OK;
    const auto natural = [](const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
    if (u->counts) {
        if (!u->slot) return W4_ERR_NULL;
        if (u->slots < 1 || u->counts_stride < N) return W4_ERR_SHAPE;
        if (!natural(u->counts, 2) || !natural(u->slot, 4) || !natural(u->repetition, 4) || !natural(u->presence, 4) ||
            !natural(u->frequency, 4))
            return W4_ERR_ALIGN;
        r.counts = u->counts;
        r.stride = u->counts_stride;
        r.slots = u->slots;
        r.slot = u->slot;
        r.rep = u->repetition;
        r.pres = u->presence;
        r.freq = u->frequency;
        r.vec = aligned16(u->counts) && u->counts_stride % 8 == 0;
    }
    if (u->bias_offsets) {
        if (!u->bias_tokens || !u->bias_values) return W4_ERR_NULL;
        if (u->bias_entries < 0 || u->bias_entries > 1 << 30) return W4_ERR_SHAPE;
        if (!natural(u->bias_offsets, 4) || !natural(u->bias_tokens, 4) || !natural(u->bias_values, 4))
            return W4_ERR_ALIGN;
        r.boff = u->bias_offsets;
        r.btok = u->bias_tokens;
        r.bval = u->bias_values;
        r.entries = u->bias_entries;
    }
    if (u->allowed) {
        if (u->allowed_stride < (N + 31) / 32) return W4_ERR_SHAPE;
        if (!natural(u->allowed, 4)) return W4_ERR_ALIGN;
        r.allowed = reinterpret_cast<const uint8_t *>(u->allowed);
        r.astride = 4 * u->allowed_stride;
    }
    r.on = r.counts || r.boff || r.allowed;
    return W4A16_OK;
}

}  // namespace w4a16
