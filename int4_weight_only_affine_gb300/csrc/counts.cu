// w4_token_counts: the tokens that requests have seen, counted in one row of
// 16 bits a token for each request's slot: bit 15 "in the prompt", the low 15
// bits how often it is in the output (saturating), as the penalties of
// lm_head_argmax_topk_rules read them.
//
// New tokens of running requests (add_kernel): a thread to a token finds its
// sequence by a binary search of the offsets and changes its entry with a 16-bit
// compare-and-swap, which is exact at any number of equal tokens; lanes that
// hold the same entry let the first of them do it for all.  Entries are whole
// numbers, so the order of the updates does not show.  Further blocks look the
// sequences over, for those that no token leads to.  A call is one chain of
// three or four dependent reads: 2 to 3 us, whatever it counts.
//
// New requests (reset_kernel): a block owns 8192 tokens of one slot's row, counts
// its share of the sequence's tokens in shared memory and writes the row once,
// so that clearing costs no pass of its own.  Every block of a row reads the
// sequence's tokens (from L2); the row's write bounds the call.  Blocks of half
// and twice the tokens were measured 10 % and 25 % slower (16 rows of 151936
// and 20900 tokens: 3.8 us).  Long prompts are read 2048 tokens at a time by each
// block: two of 16384, 65536 and 131072 tokens take 6.6, 20 and 39 us.
#include "common.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = 8192;  // entries of a block
constexpr uint32_t kPromptBit = 0x8000u, kMost = 0x7FFFu;

struct CountArgs {
    uint16_t *counts;
    long long stride;
    const int32_t *slot, *tokens, *offsets;
    int slots, N, batch, total, prompt;
    unsigned token_blocks;  // of add_kernel
};

// The tokens [first, end) of sequence b; false (reported) if its offsets are out of order.
__device__ __forceinline__ bool sequence(const CountArgs &a, int b, int &first, int &end) {
    first = a.offsets ? __ldg(a.offsets + b) : b;
    end = a.offsets ? __ldg(a.offsets + b + 1) : b + 1;
    if (first >= 0 && first <= end && end <= a.total) return true;
    atomicExch(&g_bad_index, 1);
    return false;
}

// The row of sequence b's slot, or null (a negative slot: none; one past the last is reported).
__device__ __forceinline__ uint16_t *row_of(const CountArgs &a, int b) {
    const int s = __ldg(a.slot + b);
    if (s >= a.slots) atomicExch(&g_bad_index, 1);
    return s >= 0 && s < a.slots ? a.counts + s * a.stride : nullptr;
}

__global__ void __launch_bounds__(kThreads) add_kernel(const CountArgs a) {
    pdl_wait();
    long long t = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (blockIdx.x >= a.token_blocks) {  // the blocks behind the tokens look the sequences over, a thread to each
        t -= (long long)a.token_blocks * kThreads;
        int first, end;
        if (t < a.batch) {
            sequence(a, (int)t, first, end);
            row_of(a, (int)t);
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    uint16_t *p = nullptr;
    if (t < a.total) {
        const int n = __ldg(a.tokens + t);
        int b = (int)t;
        if (a.offsets) {  // the last sequence that begins at t or before
            int lo = -1, hi = a.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (__ldg(a.offsets + mid) <= t) lo = mid;
                else hi = mid;
            }
            b = lo;
        }
        int first, end;
        if (b >= 0 && sequence(a, b, first, end) && t >= first && t < end) {
            uint16_t *row = row_of(a, b);
            if (n >= a.N) atomicExch(&g_bad_index, 1);
            if (row && n >= 0 && n < a.N) p = row + n;
        }
    }
    // (A lane without an entry matches none: its key is odd, entries are even.)
    const unsigned long long key = p ? reinterpret_cast<unsigned long long>(p) : 2ull * lane + 1ull;
    const unsigned same = __match_any_sync(~0u, key);
    if (!p || (same & ((1u << lane) - 1u)) != 0u) return;
    const uint32_t add = __popc(same);
    unsigned short old = *reinterpret_cast<volatile unsigned short *>(p);
    while (true) {
        const uint32_t c = old;
        const uint32_t now = a.prompt ? c | kPromptBit : (c & kPromptBit) | min((c & kMost) + add, kMost);
        if (now == c) break;
        const unsigned short was = atomicCAS(reinterpret_cast<unsigned short *>(p), old, (unsigned short)now);
        if (was == old) break;
        old = was;
    }
}

__global__ void __launch_bounds__(kThreads) reset_kernel(const CountArgs a) {
    __shared__ __align__(16) uint32_t seen[kSpan];  // bit 31: in the prompt; the rest: times in the output
    pdl_wait();
    const int b = blockIdx.y, lo = blockIdx.x * kSpan, span = min(kSpan, a.N - lo);
    int first, end;
    const bool ordered = sequence(a, b, first, end);
    uint16_t *row = row_of(a, b);
    if (!row) return;
    bool taken = false;  // by a later sequence: the row is that one's
    for (int i = b + 1 + threadIdx.x; i < a.batch; i += kThreads) taken |= __ldg(a.slot + i) == __ldg(a.slot + b);
    for (int i = threadIdx.x; i < kSpan / 4; i += kThreads) reinterpret_cast<uint4 *>(seen)[i] = make_uint4(0, 0, 0, 0);
    if (__syncthreads_or(taken)) {
        if (threadIdx.x == 0) atomicExch(&g_bad_index, 1);
        return;
    }
    if (ordered) {
        constexpr int kAhead = 8;
        for (int at = first; at < end; at += kAhead * kThreads) {
            int n[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = at + j * kThreads + (int)threadIdx.x;
                n[j] = i < end && i >= at ? __ldg(a.tokens + i) : -1;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (n[j] >= a.N) atomicExch(&g_bad_index, 1);
                if (n[j] >= lo && n[j] < lo + span) {
                    if (a.prompt) atomicOr(seen + (n[j] - lo), 1u << 31);
                    else atomicAdd(seen + (n[j] - lo), 1u);
                }
            }
            if (end - at <= kAhead * kThreads) break;  // (at would pass 2^31)
        }
    }
    __syncthreads();
    const auto entry = [&](int i) { return (seen[i] >> 16 & kPromptBit) | min(seen[i] & 0x7FFFFFFFu, kMost); };
    uint16_t *dst = row + lo;
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(dst) & 15u) == 0) {
        done = span / 8 * 8;
        for (int i = 8 * threadIdx.x; i < done; i += 8 * kThreads) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = entry(i + 2 * j) | entry(i + 2 * j + 1) << 16;
            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    for (int i = done + threadIdx.x; i < span; i += kThreads) dst[i] = (uint16_t)entry(i);
}

}  // namespace

// Reads and clears this translation unit's record of bad indexes.
int counts_bad_index() {
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

extern "C" int w4_token_counts(uint16_t *counts, int64_t counts_stride, int slots, int N, const int32_t *slot,
                               const int32_t *tokens, const int32_t *offsets, int batch, int total, unsigned flags,
                               void *stream) {
    if (!counts || (!slot && batch != 0)) return W4_ERR_NULL;  // (an empty array may have no address)
    if (slots < 1 || N < 1 || counts_stride < N || batch < 0 || total < 0 || (!offsets && total != batch) ||
        batch > 65535 || (flags & ~(unsigned)(W4_COUNTS_PROMPT | W4_COUNTS_RESET)) != 0)
        return W4_ERR_SHAPE;
    if (total > 0 && !tokens) return W4_ERR_NULL;
    if (((reinterpret_cast<uintptr_t>(slot) | reinterpret_cast<uintptr_t>(tokens) |
          reinterpret_cast<uintptr_t>(offsets)) & 3u) != 0 || (reinterpret_cast<uintptr_t>(counts) & 1u) != 0)
        return W4_ERR_ALIGN;
    const bool reset = (flags & W4_COUNTS_RESET) != 0;
    if (batch == 0 || (total == 0 && !reset)) return W4A16_OK;
    if (device_cc() != 103) return W4_ERR_DEVICE;
    const CountArgs a{counts, counts_stride, slot, tokens, offsets, slots, N, batch, total,
                      (flags & W4_COUNTS_PROMPT) != 0, (unsigned)((total + (long long)kThreads - 1) / kThreads)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = reset ? dim3((unsigned)((N + (long long)kSpan - 1) / kSpan), (unsigned)batch, 1)
                        : dim3(a.token_blocks + (offsets ? (unsigned)((batch + kThreads - 1) / kThreads) : 0u), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, reset ? reset_kernel : add_kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return W4_ERR_LAUNCH;
    }
    return W4A16_OK;
}
