// Rules of token selection (w4_logit_rules): penalties of tokens that a request
// has seen, biases of listed tokens, and a mask, applied to the fp32 logits of a
// block's rows while they lie in shared memory, before the block selects from
// them.
//
// For logit l of token n in row m, with c = counts[slot[m]][n]:
//     c != 0:            z = l > 0 ? l / repetition : l * repetition
//     t = c & 0x7FFF:    z = z - frequency * t;   t != 0: z = z - presence
//     biases:            z = z + value, for each of the row's entries for n in the list's order
//     mask bit 0:        n cannot be selected
// each step one fp32 operation, rounded to nearest.  The rules read 2 bytes of
// counts and a bit of mask per logit, against the 0.5625 K bytes of weight that
// made it: they are bound by the latency of these reads, which a block therefore
// asks into L2 while it still streams weights, and issues several at a time.
// 151936 tokens: one row, K 1024, penalties, 24.4 us for 22.5 without; 16 rows, K 2048,
// penalties, 300 biases a row and a mask, top 50, 105 us for 91.1.  Every block reads
// all lists of biases, by one warp: with 1000, 3000 and 10000 entries a row these no
// longer hide behind the stream (124, 261 and 707 us).
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
    int most;  // biases in the block's tokens that there is room for: kMaxHits, or none without biases
};

// What stands in place of a masked logit: a NaN that no operation makes.
constexpr uint32_t kExcluded = 0xFFFFFFFFu;

// What a block keeps of each row while it streams weights: its place in the counts
// (-1: no penalties), its penalties and its list of biases.
struct RowRule {
    long long counts;
    float rep, pres, freq;
    int b0, b1;
};
// A bias that falls into the block's tokens: row and place in its list, token.
struct BiasHit {
    int m, at, token;
    float value;
};
constexpr int kMaxHits = 256;  // more of them are left to the warps, one list after the other

// The block's memory of the rules: rows, hits and their number.
inline size_t rules_bytes(const Rules &r, int M) { return 16 + M * sizeof(RowRule) + r.most * sizeof(BiasHit); }
struct RulesMemory {
    RowRule *rule;
    BiasHit *hits;
    int *nhits;
    __device__ __forceinline__ RulesMemory(uint8_t *p, int M)
        : rule(reinterpret_cast<RowRule *>(p + 16)), hits(reinterpret_cast<BiasHit *>(p + 16 + M * sizeof(RowRule))),
          nhits(reinterpret_cast<int *>(p)) {}
};

// Done by one warp of its own while the others stream weights (after that, where shared
// memory is short): reads the rows' rules, asks the counts and masks of tokens n0 .. n0 + rows - 1 into L2, and
// searches the lists of biases for these tokens.  M <= 16.
__device__ __forceinline__ void rules_begin(const Rules &r, const RulesMemory &k, int M, int N, int n0, int rows,
                                            int lane) {
    RowRule v{-1, 1.f, 0.f, 0.f, 0, 0};
    if (lane < M) {
        const int s = r.counts ? __ldg(r.slot + lane) : -1;
        v.rep = r.counts && r.rep ? __ldg(r.rep + lane) : 1.f;
        v.pres = r.counts && r.pres ? __ldg(r.pres + lane) : 0.f;
        v.freq = r.counts && r.freq ? __ldg(r.freq + lane) : 0.f;
        if (r.boff) {
            v.b0 = __ldg(r.boff + lane);
            v.b1 = __ldg(r.boff + lane + 1);
        }
        const bool list = v.b0 >= 0 && v.b0 <= v.b1 && v.b1 <= r.entries;
        if (!list) v.b0 = v.b1 = 0;
        if (s >= 0 && s < r.slots) v.counts = s * r.stride;
        if (!list || (r.counts && s >= r.slots)) atomicExch(&g_bad_index, 1);
        k.rule[lane] = v;
    }
    const int lines = (rows + 63) / 64;  // of 128 bytes: 64 counts, 1024 mask bits
    for (int m = 0; m < M; ++m) {
        const long long at = __shfl_sync(~0u, v.counts, m);
        for (int l = lane; l < lines; l += 32) {
            const int n = n0 + 64 * l;
            if (at >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(r.counts + at + n));
            if (r.allowed && l % 16 == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(r.allowed + m * r.astride + n / 8));
        }
    }
    int found = 0;
    for (int m = 0; m < M; ++m) {
        const int end = __shfl_sync(~0u, v.b1, m);
        for (int at = __shfl_sync(~0u, v.b0, m); at < end; at += 256) {
            int tok[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) tok[q] = at + 32 * q + lane < end ? __ldg(r.btok + at + 32 * q + lane) : -1;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (tok[q] >= N) atomicExch(&g_bad_index, 1);
                const bool mine = tok[q] >= n0 && tok[q] < n0 + rows;
                const unsigned bal = __ballot_sync(~0u, mine);
                const int h = found + __popc(bal & ((1u << lane) - 1u)), i = at + 32 * q + lane;
                if (mine && h < r.most) k.hits[h] = BiasHit{m, i, tok[q], __ldg(r.bval + i)};
                found += __popc(bal);  // (hits lie in the order of their lists)
            }
        }
    }
    if (lane == 0) *k.nhits = found;
}

// Biases of row m, by one warp: 32 entries at a time; the first lane of a token
// adds all of that token in the chunk to its logit, in order.
__device__ __noinline__ void rules_biases_in_order(const Rules &r, float *z, int n0, int rows, int o0, int o1, int lane) {
    for (int at = o0; at < o1; at += 32) {
        const int tok = at + lane < o1 ? __ldg(r.btok + at + lane) : -1;
        const bool mine = tok >= n0 && tok < n0 + rows;
        if (!__any_sync(~0u, mine)) continue;
        const float v = mine ? __ldg(r.bval + at + lane) : 0.f;
        const unsigned same = __match_any_sync(~0u, mine ? tok : -1 - lane);
        const float old = mine ? z[tok - n0] : 0.f;
        float sum = old;
        for (int l = 0; l < 32; ++l) {
            const float w = __shfl_sync(~0u, v, l);
            if (same >> l & 1u) sum = __fadd_rn(sum, w);
        }
        __syncwarp();  // (every lane has read its logit)
        if (mine && (same & ((1u << lane) - 1u)) == 0u && __float_as_uint(old) != kExcluded) z[tok - n0] = sum;
        __syncwarp();
    }
}

// The logits res[m * ld + i] of tokens n0 + i, i < rows (n0 a multiple of 16),
// under the rules.  Called by every thread of the block, with a barrier before;
// ends with one.
__device__ __forceinline__ void rules_apply(const Rules &r, const RulesMemory &k, float *res, int ld, int M, int n0,
                                            int rows, int tid, int threads) {
    // Eight tokens of one row of logits a thread: 16 bytes of counts, a byte of mask;
    // the reads of four such units at a time.  e / M = e * by >> 20 while e < 2^16
    // (a block holds far fewer).
    const int units = (rows + 7) / 8 * M, by = ((1 << 20) + M - 1) / M;
    constexpr int kAhead = 4;
    for (int e0 = r.counts || r.allowed ? tid : units; e0 < units; e0 += kAhead * threads) {
        uint4 c[kAhead];
        uint32_t bits[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int e = e0 + q * threads, g = (int)((long long)e * by >> 20), m = e - g * M, i0 = 8 * g;
            c[q] = make_uint4(0u, 0u, 0u, 0u);
            bits[q] = 0xFFu;
            if (e >= units) continue;
            if (r.allowed) bits[q] = __ldg(r.allowed + m * r.astride + (n0 + i0) / 8);
            const long long at = k.rule[m].counts;
            if (at < 0) continue;
            const uint16_t *src = r.counts + at + n0 + i0;
            if (r.vec && rows - i0 >= 8) {
                c[q] = __ldg(reinterpret_cast<const uint4 *>(src));
            } else {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = i0 + j < rows ? __ldg(src + j) : 0;
                c[q] = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
            }
        }
#pragma unroll 1
        for (int q = 0; q < kAhead; ++q) {
            const int e = e0 + q * threads, g = (int)((long long)e * by >> 20), m = e - g * M, i0 = 8 * g;
            // (One of four without an index, so that the copies stay in registers.)
            const uint4 n4 = q == 0 ? c[0] : q == 1 ? c[1] : q == 2 ? c[2] : c[3];
            const uint32_t bit = q == 0 ? bits[0] : q == 1 ? bits[1] : q == 2 ? bits[2] : bits[3];
            if (e >= units || ((n4.x | n4.y | n4.z | n4.w) == 0u && bit == 0xFFu)) continue;
            float *p = res + m * ld + i0;
            const uint32_t w[4] = {n4.x, n4.y, n4.z, n4.w};
            uint32_t seen = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu) seen |= 1u << j;
                if (!(bit >> j & 1u) && i0 + j < rows) p[j] = __uint_as_float(kExcluded);
            }
            seen &= bit;
            const float rep = k.rule[m].rep, pres = k.rule[m].pres, freq = k.rule[m].freq;
            while (seen) {  // (few of eight)
                const int j = __ffs(seen) - 1;
                seen &= seen - 1u;
                const uint32_t two = j < 2 ? w[0] : j < 4 ? w[1] : j < 6 ? w[2] : w[3];
                const int t = two >> (16 * (j & 1)) & 0x7FFF;
                float z = p[j];
                z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                if (t) z = __fsub_rn(__fsub_rn(z, __fmul_rn(freq, (float)t)), pres);
                p[j] = z;
            }
        }
    }
    __syncthreads();
    if (!r.boff) return;
    const int n = *k.nhits;
    if (n <= r.most) {
        // The first hit of a token adds all of that token to its logit, in their order (as the
        // other branch does: the result must not depend on how many hits a block has).
        for (int h = tid; h < n; h += threads) {
            const BiasHit b = k.hits[h];
            bool first = true;
            for (int i = 0; i < h; ++i) first = first && (k.hits[i].m != b.m || k.hits[i].token != b.token);
            if (!first) continue;
            float *p = res + b.m * ld + (b.token - n0);
            float z = *p;
            if (__float_as_uint(z) == kExcluded) continue;
            z = __fadd_rn(z, b.value);
            for (int i = h + 1; i < n; ++i)
                if (k.hits[i].m == b.m && k.hits[i].token == b.token) z = __fadd_rn(z, k.hits[i].value);
            *p = z;
        }
    } else {
        for (int m = tid >> 5; m < M; m += threads >> 5)
            rules_biases_in_order(r, res + m * ld, n0, rows, k.rule[m].b0, k.rule[m].b1, tid & 31);
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
    r.most = r.boff ? kMaxHits : 0;
    return W4A16_OK;
}

}  // namespace w4a16
