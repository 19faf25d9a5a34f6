// What the calls on the paged key/value cache share: a sequence's place in a
// batch, read from the device arrays, and the host checks of the public structs.
#pragma once

#include "common.cuh"

namespace w4a16 {

constexpr int kMaxHeads = 1024;

// Division of 0 <= n < 2^31 by a d fixed on the host: with l = ceil(log2 d)
// and m = ceil(2^(31 + l) / d) < 2^32, floor(n m / 2^(31 + l)) is floor(n / d),
// since m exceeds 2^(31 + l) / d by less than 1 <= 2^l / d and n < 2^31.
struct FastDiv {
    uint32_t d, m, shift;
};
inline FastDiv fast_div(int d) {
    uint32_t l = 0;
    while ((1ull << l) < (uint64_t)d) ++l;
    return FastDiv{(uint32_t)d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}
__device__ __forceinline__ int operator/(int n, const FastDiv &f) {
    return (int)(((uint64_t)(uint32_t)n * f.m) >> f.shift);
}
__device__ __forceinline__ int operator%(int n, const FastDiv &f) { return n - n / f * (int)f.d; }

struct KvBatch {
    const int32_t *table, *q_offsets, *kv_lens;
    int batch, max_pages, table_stride, total_q;
    int max_kv;  // max_pages * page_size, at most INT_MAX
};

// One sequence: its first token, its number of new tokens and its tokens in
// the cache, clamped to the tensors' sizes.
struct Seq {
    int q0, qn, kv;
    bool ordered;  // the offsets ascend, within the tensors
    bool fits;     // the length is one that the table has room for
};

__device__ __forceinline__ Seq load_seq(const KvBatch &b, int i) {
    const int o0 = __ldg(b.q_offsets + i), o1 = __ldg(b.q_offsets + i + 1), kv = __ldg(b.kv_lens + i);
    Seq s;
    s.q0 = min(max(o0, 0), b.total_q);
    s.qn = min(max(o1, s.q0), b.total_q) - s.q0;
    s.kv = min(max(kv, 0), b.max_kv);
    s.ordered = s.q0 == o0 && s.q0 + s.qn == o1;
    s.fits = s.kv == kv;
    if (!s.ordered || !s.fits) atomicExch(&g_bad_index, 1);
    return s;
}

inline bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0; }

// Host checks of a batch; fills the device form.
inline int check_batch(const f16_kv_batch *b, int page_size, KvBatch &out) {
    if (!b || !b->block_table || !b->q_offsets || !b->kv_lens) return W4_ERR_NULL;
    if (b->batch < 1 || b->max_pages < 1 || b->table_stride < b->max_pages || b->total_q < 0 || b->max_q_len < 0)
        return W4_ERR_SHAPE;
    if (((reinterpret_cast<uintptr_t>(b->block_table) | reinterpret_cast<uintptr_t>(b->q_offsets) |
          reinterpret_cast<uintptr_t>(b->kv_lens)) & 3u) != 0)
        return W4_ERR_ALIGN;
    const long long most = (long long)b->max_pages * page_size;
    out.table = b->block_table;
    out.q_offsets = b->q_offsets;
    out.kv_lens = b->kv_lens;
    out.batch = b->batch;
    out.max_pages = b->max_pages;
    out.table_stride = b->table_stride;
    out.total_q = b->total_q;
    out.max_kv = most < 0x7FFFFFFFll - 4096 ? (int)most : 0x7FFFFFFF - 4096;
    return W4A16_OK;
}

inline bool head_dim_ok(int d) { return d >= 8 && d <= 256 && d % 8 == 0; }

// Positions of a key tile of the kernels for this head_dim (at most).
__host__ __device__ constexpr int kv_tile(int head_dim) { return head_dim <= 128 ? 128 : 64; }

// Rows of one copy from the cache: the largest power of two that divides the
// page, up to a tile (8 rows are one swizzle atom, so every copy starts on one).
inline int kv_box_rows(int page_size, int head_dim) {
    int r = 8;
    while (r < kv_tile(head_dim) && page_size % (2 * r) == 0) r *= 2;
    return r;
}

inline int check_cache(const f16_kv_cache *c) {
    if (!c || !c->k || !c->v) return W4_ERR_NULL;
    if (c->num_pages < 1 || c->page_size < 8 || c->page_size % 8 != 0 || c->heads < 1 || c->heads > kMaxHeads ||
        !head_dim_ok(c->head_dim) || c->box_rows != kv_box_rows(c->page_size, c->head_dim))
        return W4_ERR_SHAPE;
    return W4A16_OK;
}

}  // namespace w4a16
