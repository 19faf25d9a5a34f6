"""f16_attention against the binary64 oracle: head layouts, lengths from one
token to long ones, pages that end inside a tile, windows, rows that see
nothing, and whatever the cache holds where nobody looks."""
import numpy as np
import pytest

from _attn import Batch, attention
from _gpu import require_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    return w4


def data(batch, hq, hkv, d, seed, garbage=True):
    """q, k_cache, v_cache in binary16; cache slots of no position are NaN and infinities."""
    g = np.random.RandomState(seed)
    q = (g.standard_normal((batch.tokens, hq, d)) * np.exp2(g.uniform(-1, 1.5, (1, hq, 1)))).astype(np.float16)
    kc, vc = (g.standard_normal((batch.pages, batch.page, hkv, d)).astype(np.float16) for _ in range(2))
    if garbage:
        free = ~batch.used()
        kc[free], vc[free] = np.nan, np.inf
    return q, kc, vc


def device_batch(w4, batch, max_q=None):
    return w4.KVBatch(to_dev(batch.table), to_dev(batch.offsets), to_dev(batch.kv_lens.astype(np.int32)),
                      batch.tokens, int(batch.q_lens.max()) if max_q is None else max_q)


def check(got, want, tol, what):
    got = got.cpu().numpy().astype(np.float64)
    inside = ~np.isnan(want)
    fin = inside & np.isfinite(want)
    assert np.array_equal(got[inside & ~fin], want[inside & ~fin]), what
    err = np.abs(got[fin] - want[fin])
    assert np.all(err <= tol[fin]), (what, float((err / tol[fin]).max()))


def run(w4, batch, hq, hkv, d, causal=True, window=0, scale=None, seed=0, max_q=None, garbage=True):
    import torch
    q, kc, vc = data(batch, hq, hkv, d, seed, garbage)
    cache = w4.KVCache(to_dev(kc), to_dev(vc))
    y = torch.full((batch.tokens, hq, d), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((batch.tokens, hq), 7.0, dtype=torch.float32, device="cuda")
    kb = device_batch(w4, batch, max_q)
    ws = w4.attention_workspace(cache, hq, kb.max_q_len)
    ws[2064:] = 255   # NaN past the counters: what an earlier call left there may not matter
    w4.f16_attention(to_dev(q), cache, kb, y=y, lse=lse, scale=scale, causal=causal, window=window, workspace=ws)
    assert w4.device_status() == 0
    assert not bool(ws[:2048].any())   # the counts of parts are ready for the next call
    sc = d**-0.5 if scale is None else scale
    wy, wl, ty, tl = attention(q, kc, vc, batch, sc, causal, window)
    check(y, wy, ty, "y")
    check(lse, wl, tl, "lse")
    outside = slice(int(batch.offsets[-1]), None)   # rows of no sequence keep what they held
    assert bool((y[outside] == 7.0).all()) and bool((lse[outside] == 7.0).all())
    return y, lse


HEADS = [(1, 1, 64), (16, 2, 128), (16, 8, 128), (14, 2, 64), (6, 6, 128), (5, 1, 72), (20, 1, 64), (40, 2, 8),
         (4, 2, 80), (12, 4, 96), (8, 2, 136), (4, 1, 192), (3, 1, 200), (8, 4, 256)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_single_tokens_by_head_layout(w4, hq, hkv, d):
    run(w4, Batch([1] * 6, [1, 5, 128, 129, 300, 777], 16, seed=d), hq, hkv, d)


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_chunks_by_head_layout(w4, hq, hkv, d):
    run(w4, Batch([37, 1, 130, 2], [37, 260, 333, 5], 16, seed=d), hq, hkv, d)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 96, 128, 256, 1000])
def test_page_sizes(w4, page):
    run(w4, Batch([1, 3, 70, 200], [260, 131, 197, 200], page, seed=page), 16, 2, 128)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 513])
def test_prompt_lengths(w4, n):
    run(w4, Batch([n], [n], 16, seed=n), 16, 2, 128)
    run(w4, Batch([n], [n], 16, seed=n), 14, 2, 64)


@pytest.mark.parametrize("q,kv", [(1, 4097), (2, 5000), (4, 3001), (8, 2500), (16, 2049), (33, 6000), (64, 4099), (150, 3333)])
def test_chunk_over_long_context(w4, q, kv):
    """One sequence shared out over the whole GPU: items of many parts."""
    run(w4, Batch([q], [kv], 32, seed=q), 16, 2, 128)
    run(w4, Batch([q], [kv], 16, seed=q), 7, 1, 64)


def test_long_context_single_token(w4):
    run(w4, Batch([1], [70001], 64, seed=1), 16, 8, 128)
    run(w4, Batch([1, 1], [50000, 3], 64, seed=2), 8, 8, 64)


@pytest.mark.parametrize("window", [1, 2, 16, 100, 128, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(w4, window, causal):
    run(w4, Batch([1, 90, 300, 5], [700, 400, 300, 2000], 16, seed=window), 16, 2, 128, causal, window)
    run(w4, Batch([1, 90, 300, 5], [700, 400, 300, 2000], 16, seed=window), 14, 2, 64, causal, window)


def test_not_causal(w4):
    run(w4, Batch([1, 77, 256, 19], [100, 77, 600, 1000], 32, seed=4), 16, 8, 128, causal=False)


def test_evicted_pages_before_a_window(w4):
    """Pages wholly before every window may be gone: no page in the table, garbage in the slots."""
    import torch
    batch = Batch([1, 40], [900, 700], 16, seed=8)
    q, kc, vc = data(batch, 16, 2, 128, 8)
    wy, wl, ty, tl = attention(q, kc, vc, batch, 128**-0.5, True, 100)
    for b in range(2):
        first = int(batch.kv_lens[b] - batch.q_lens[b] - 100 + 1)   # the first position anybody sees
        gone = np.arange(first // 16)
        pages = batch.table[b, gone].copy()
        kc[pages], vc[pages] = np.nan, np.nan
        p, at = batch.slot(b, np.arange(first))
        kc[p, at], vc[p, at] = np.inf, np.nan
        batch.table[b, gone] = 10**6 + b
    cache = w4.KVCache(to_dev(kc), to_dev(vc))
    y = w4.f16_attention(to_dev(q), cache, device_batch(w4, batch), window=100)
    assert w4.device_status() == 0
    check(y, wy, ty, "y")


def test_rows_that_see_nothing(w4):
    """Padded slots (no token cached), sequences without new tokens, and more new tokens than cached ones."""
    for mq in (None, 200):   # mixed with long chunks, or not
        y, lse = run(w4, Batch([1, 0, 1, 5, 0, 3], [0, 50, 20, 2, 0, 0], 16, seed=3, extra_rows=2), 16, 2, 128, max_q=mq)
        assert bool((y[0] == 0).all()) and bool((lse[0] == -float("inf")).all())
        assert bool((y[2:5] == 0).all())   # tokens at positions -3, -2, -1
    run(w4, Batch([300, 0, 1], [40, 50, 0], 16, seed=3, extra_rows=2), 16, 2, 128)
    run(w4, Batch([300, 0, 1], [40, 50, 0], 16, seed=3, extra_rows=2), 16, 2, 128, causal=False)


def test_no_tokens_at_all(w4):
    import torch
    batch = Batch([0, 0], [40, 0], 16, seed=3)
    _, kc, vc = data(batch, 2, 1, 64, 0)
    cache = w4.KVCache(to_dev(kc), to_dev(vc))
    y = w4.f16_attention(torch.empty(0, 2, 64, dtype=torch.float16, device="cuda"), cache, device_batch(w4, batch))
    assert y.shape == (0, 2, 64)
    run(w4, Batch([0, 0], [40, 0], 16, seed=3, extra_rows=3), 2, 1, 64)


@pytest.mark.parametrize("n", [200, 700, 3000])
def test_many_sequences(w4, n):
    g = np.random.RandomState(n)
    ql = (g.rand(n) < 0.9).astype(int)
    kl = np.maximum(g.randint(0, 80, n), ql)
    run(w4, Batch(ql, kl, 8, seed=n), 2, 1, 64)
    ql = np.where(g.rand(n) < 0.02, g.randint(1, 60, n), ql)
    kl = np.maximum(kl, ql)
    run(w4, Batch(ql, kl, 8, seed=n), 2, 1, 64, max_q=64)


@pytest.mark.parametrize("q", [1, 8, 70])
@pytest.mark.parametrize("n,kv", [(16, [300]), (24, [300]), (40, [600]), (16, [1200]), (16, [1200, 1000, 1100, 1190]),
                                  (12, [2000, 70, 1, 900]), (64, [150, 700, 90])])
def test_items_left_whole_or_cut(w4, q, n, kv):
    """About as many items as the GPU has blocks, alike or not, with empty sequences among them."""
    ql = [0 if i % 5 == 3 else q for i in range(n)]
    kl = [max(kv[i % len(kv)], ql[i]) for i in range(n)]
    run(w4, Batch(ql, kl, 16, seed=n + q), 16, 4, 128)
    run(w4, Batch(ql, kl, 16, seed=n + q), 28, 4, 64)
    if q < 70:
        run(w4, Batch(ql, kl, 16, seed=n + q), 4, 2, 256)


@pytest.mark.parametrize("ql,kl,hq,hkv,d,causal", [
    ([600] * 6, [600] * 6, 16, 8, 128, True), ([1300, 700, 0, 900, 1300, 40, 1000], [1300, 750, 9, 900, 2000, 40, 1000], 16, 8, 128, True),
    ([700, 650, 0, 655], [700, 900, 0, 655], 28, 4, 64, True), ([2100], [2100], 32, 8, 128, True),
    ([900] * 5, [900] * 5, 16, 4, 64, False), ([1, 1200, 1200, 1, 1200], [50, 1200, 1200, 2000, 1300], 16, 8, 128, True)])
def test_items_from_a_queue(w4, ql, kl, hq, hkv, d, causal):
    """More items than blocks, none costlier than an even share: taken whole, and the same whoever takes them."""
    import torch
    batch = Batch(ql, kl, 16, seed=len(ql), extra_rows=3)
    y, lse = run(w4, batch, hq, hkv, d, causal)
    q, kc, vc = data(batch, hq, hkv, d, 0)
    cache, kb = w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    ws = w4.attention_workspace(cache, hq, kb.max_q_len)
    for _ in range(5):
        y2 = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
        w4.f16_attention(to_dev(q), cache, kb, y=y2, causal=causal, workspace=ws)
        assert bool((y == y2).all()) and not bool(ws[:2048].any()) and not bool(ws[2056:2064].any())
    assert w4.device_status() == 0


def test_max_q_len_is_a_hint(w4):
    """Results hold whatever max_q_len says."""
    for hint in (0, 1, 5, 10**6):
        run(w4, Batch([1, 200, 3], [50, 230, 400], 16, seed=6), 16, 2, 128, max_q=hint)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 3.0])
def test_scales(w4, scale):
    """Flat and sharp softmaxes (scores of hundreds at scale 3)."""
    run(w4, Batch([1, 140], [900, 500], 16, seed=5), 16, 2, 128, scale=scale)


def test_rising_scores(w4):
    """Scores that grow along the context move the running maximum in every tile."""
    import torch
    batch = Batch([1, 260], [3000, 1500], 16, seed=5)
    q, kc, vc = data(batch, 8, 1, 128, 5)
    q = np.abs(q)
    for b in range(2):
        p, at = batch.slot(b, np.arange(batch.kv_lens[b]))
        kc[p, at, 0] = (np.arange(batch.kv_lens[b]) / 700.0)[:, None].astype(np.float16)
    y = w4.f16_attention(to_dev(q), w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch))
    wy, _, ty, _ = attention(q, kc, vc, batch, 128**-0.5)
    check(y, wy, ty, "y")


def test_strides_and_head_major_pages(w4):
    """q and y as parts of wider rows, K and V interleaved in one allocation, pages of [heads][tokens]."""
    import torch
    for ql, kl in (([1, 1], [300, 77]), ([150, 9], [400, 77])):
        batch = Batch(ql, kl, 16, seed=9)
        hq, hkv, d = 6, 3, 64
        q, kc, vc = data(batch, hq, hkv, d, 9)
        wide = torch.full((batch.tokens, hq + 2, d + 16), 5.0, dtype=torch.float16, device="cuda")
        wide[:, 1:-1, 8:-8] = to_dev(q)
        both = torch.zeros(batch.pages, 2, hkv, 16, d, dtype=torch.float16, device="cuda")
        both[:, 0] = to_dev(kc).transpose(1, 2)
        both[:, 1] = to_dev(vc).transpose(1, 2)
        cache = w4.KVCache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
        out = torch.full((hq + 1, batch.tokens, d), 5.0, dtype=torch.float16, device="cuda")
        y = w4.f16_attention(wide[:, 1:-1, 8:-8], cache, device_batch(w4, batch), y=out[1:].transpose(0, 1))
        wy, _, ty, _ = attention(q, kc, vc, batch, d**-0.5)
        check(y, wy, ty, "y")
        assert bool((out[0] == 5.0).all())
        # in place: y over q
        qq = to_dev(q)
        w4.f16_attention(qq, cache, device_batch(w4, batch), y=qq)
        check(qq, wy, ty, "y in place")


def test_results_repeat(w4):
    for ql, kl in (([1, 1, 1], [9000, 30, 700]), ([300, 20], [900, 5000])):
        batch = Batch(ql, kl, 16, seed=2)
        a, la = run(w4, batch, 16, 2, 128)
        b, lb = run(w4, batch, 16, 2, 128)
        assert bool((a == b).all()) and bool((la == lb).all())


def test_other_stream_and_captured_graph(w4):
    """A graph captured for one batch is replayed with other lengths and pages in the same tensors."""
    import torch
    hq, hkv, d = 16, 2, 128
    for ql in ([1, 1, 1], [100, 1, 30]):
        first, second = Batch(ql, [600, 2000, 37], 16, seed=1, spare=200), Batch(ql, [1100, 130, 900], 16, seed=2, spare=200)
        pages = max(first.pages, second.pages)
        g = np.random.RandomState(0)
        q = g.standard_normal((first.tokens, hq, d)).astype(np.float16)
        kc, vc = (g.standard_normal((pages, 16, hkv, d)).astype(np.float16) for _ in range(2))
        width = max(first.table.shape[1], second.table.shape[1])
        tables = [np.pad(b.table, ((0, 0), (0, width - b.table.shape[1])), constant_values=-1) for b in (first, second)]
        cache = w4.KVCache(to_dev(kc), to_dev(vc))
        table, offs, lens = to_dev(tables[0]), to_dev(first.offsets), to_dev(first.kv_lens.astype(np.int32))
        kb = w4.KVBatch(table, offs, lens, first.tokens, max(ql))
        ws = w4.attention_workspace(cache, hq, max(ql))
        tq, y = to_dev(q), torch.zeros(first.tokens, hq, d, dtype=torch.float16, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            w4.f16_attention(tq, cache, kb, y=y, workspace=ws)
        side.synchronize()
        check(y, *attention(q, kc, vc, first, d**-0.5)[0:3:2], "side stream")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w4.f16_attention(tq, cache, kb, y=y, workspace=ws)
        for b, t in ((second, tables[1]), (first, tables[0])):
            table.copy_(to_dev(t))
            lens.copy_(to_dev(b.kv_lens.astype(np.int32)))
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            check(y, *attention(q, kc, vc, b, d**-0.5)[0:3:2], "replay")
    assert w4.device_status() == 0


def test_calls_on_two_streams_at_once(w4):
    """Calls that share the GPU, each with a workspace of its own: blocks of a call that cannot all run at once."""
    import torch
    hq, hkv, d = 16, 2, 128
    cases = []
    for k, (ql, kl) in enumerate((([1, 1], [30000, 100]), ([200, 1], [9000, 3000]), ([3], [20000]), ([700], [2500]))):
        batch = Batch(ql, kl, 16, seed=k)
        q, kc, vc = data(batch, hq, hkv, d, k)
        cache, kb = w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
        want = w4.f16_attention(to_dev(q), cache, kb)
        cases.append((to_dev(q), cache, kb, want, w4.attention_workspace(cache, hq, 700), torch.cuda.Stream(),
                      [torch.empty_like(want) for _ in range(20)]))
    torch.cuda.synchronize()
    for i in range(20):
        for q, cache, kb, want, ws, stream, ys in cases:
            w4.f16_attention(q, cache, kb, y=ys[i], workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert w4.device_status() == 0
    for q, cache, kb, want, ws, stream, ys in cases:
        assert all(bool((y == want).all()) for y in ys)
        assert not bool(ws[:2048].any())


@pytest.mark.parametrize("ql,kl,hq,hkv,d", [([1, 1], [30000, 100], 16, 2, 128), ([200, 1], [9000, 3000], 16, 2, 128),
                                            ([700], [2500], 16, 2, 128), ([90, 60], [3000, 2000], 14, 2, 64),
                                            ([64], [9001], 16, 8, 128), ([2000], [2000], 8, 8, 64)])
def test_blocks_that_may_not_wait(w4, ql, kl, hq, hkv, d):
    """With a count of begun blocks that says some never began (as when another call holds part of the GPU), no
    block waits for another's part, and the last to count a part in joins them: the same bits."""
    import torch
    batch = Batch(ql, kl, 16, seed=3)
    q, kc, vc = data(batch, hq, hkv, d, 3)
    cache, kb = w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    ws = w4.attention_workspace(cache, hq, max(ql))
    lse, lse2 = (torch.empty(batch.tokens, hq, device="cuda") for _ in range(2))
    y = w4.f16_attention(to_dev(q), cache, kb, lse=lse, workspace=ws)
    ws.zero_()
    ws.view(torch.int32)[513] = 1000   # blocks begun in earlier calls, which the count of all calls lacks
    y2 = w4.f16_attention(to_dev(q), cache, kb, lse=lse2, workspace=ws)
    assert w4.device_status() == 0 and not bool(ws[:2048].any())
    assert bool((y == y2).all()) and bool((lse == lse2).all())


def test_workspace_that_was_not_zeroed(w4):
    """Waits for parts that cannot all come in run out, are reported, and the call works again on a zeroed workspace."""
    batch = Batch([1], [9000], 16, seed=5)
    q, kc, vc = data(batch, 16, 2, 128, 5)
    cache, kb = w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    ws = w4.attention_workspace(cache, 16, 1)
    ws[:1024] = 1   # counts of parts far past any item's
    w4.f16_attention(to_dev(q), cache, kb, workspace=ws)
    assert w4.device_status() == 8 and w4.device_status() == 0
    ws.zero_()
    wy, _, ty, _ = attention(q, kc, vc, batch, 128**-0.5)
    check(w4.f16_attention(to_dev(q), cache, kb, workspace=ws), wy, ty, "y")
    assert w4.device_status() == 0


@pytest.mark.parametrize("word", [514, 515])
def test_queue_that_was_not_zeroed(w4, word):
    """A queue that does not begin with its first item is reported."""
    import torch
    batch = Batch([600] * 6, [600] * 6, 16, seed=5)
    q, kc, vc = data(batch, 16, 8, 128, 5)
    cache, kb = w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    ws = w4.attention_workspace(cache, 16, 600)
    ws.view(torch.int32)[word] = 1000
    w4.f16_attention(to_dev(q), cache, kb, workspace=ws)
    assert w4.device_status() == 8 and w4.device_status() == 0
    ws.zero_()
    wy, _, ty, _ = attention(q, kc, vc, batch, 128**-0.5)
    check(w4.f16_attention(to_dev(q), cache, kb, workspace=ws), wy, ty, "y")
    assert w4.device_status() == 0


def test_offsets_past_32_bits(w4):
    """Pages that lie beyond 2**32 elements of the cache."""
    import torch
    page, hkv, d = 64, 2, 128
    pages = 2**32 // (page * hkv * d) + 64
    if torch.cuda.mem_get_info()[0] < 4 * 2**32 + 2**31:
        pytest.skip("not enough device memory")
    kc, vc = (torch.empty(pages, page, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    for ql, kl in (([1, 1], [500, 130]), ([90, 4], [500, 130])):
        batch = Batch(ql, kl, page, seed=3, spare=0)
        q, k, v = data(batch, 16, hkv, d, 3)
        far = pages - 1 - np.arange(batch.pages)
        for i in range(batch.pages):
            kc[far[i]], vc[far[i]] = to_dev(k[i]), to_dev(v[i])
        table = np.where(batch.table >= 0, far[batch.table.clip(0)], -1).astype(np.int32)
        kb = w4.KVBatch(to_dev(table), to_dev(batch.offsets), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens, max(ql))
        y = w4.f16_attention(to_dev(q), w4.KVCache(kc, vc), kb)
        wy, _, ty, _ = attention(q, k, v, batch, d**-0.5)
        check(y, wy, ty, "y")
    del kc, vc
    torch.cuda.empty_cache()


def test_indexes_out_of_range_are_reported(w4):
    """Pages the cache does not have and lengths past the table are read as nothing and reported once."""
    for ql in ([1, 1], [200, 1]):
        batch = Batch(ql, [300, 90], 16, seed=5)
        q, kc, vc = data(batch, 16, 2, 128, 5)
        good = batch.table.copy()
        wy, _, ty, _ = attention(q, kc, vc, batch, 128**-0.5)
        cache = w4.KVCache(to_dev(kc), to_dev(vc))
        batch.table[0, 3] = batch.pages       # one past the end
        batch.table[0, 5] = -1
        y = w4.f16_attention(to_dev(q), cache, device_batch(w4, batch))
        assert w4.device_status() == 9 and w4.device_status() == 0
        batch.table = good
        batch.kv_lens = batch.kv_lens + np.array([10**6, 0])
        w4.f16_attention(to_dev(q), cache, device_batch(w4, batch))
        assert w4.device_status() == 9 and w4.device_status() == 0
        batch.kv_lens = np.array([300, 90])
        # the other sequence was not touched by its neighbour's bad page
        s = slice(int(batch.offsets[1]), None)
        check(y[s], wy[s], ty[s], "neighbour")
        check(w4.f16_attention(to_dev(q), cache, device_batch(w4, batch)), wy, ty, "good again")
        bad = batch.offsets.copy()
        bad[1] = 10**6
        kb = w4.KVBatch(to_dev(batch.table), to_dev(bad), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens, max(ql))
        w4.f16_attention(to_dev(q), cache, kb)
        assert w4.device_status() == 9


@pytest.mark.parametrize("q", [1, 60])
def test_offsets_out_of_order_compute_nothing(w4, q):
    """Offsets that fall are reported, and no row is written: no plan holds for them."""
    import torch
    batch = Batch([q] * 8, [100 + q] * 8, 16, seed=3)
    x, kc, vc = data(batch, 16, 2, 128, 3)
    bad = np.array([0, batch.tokens] * 4 + [0], np.int32)
    kb = w4.KVBatch(to_dev(batch.table), to_dev(bad), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens, q)
    y = torch.full(x.shape, 7.0, dtype=torch.float16, device="cuda")
    cache = w4.KVCache(to_dev(kc), to_dev(vc))
    ws = w4.attention_workspace(cache, 16, q)
    w4.f16_attention(to_dev(x), cache, kb, y=y, workspace=ws)
    assert w4.device_status() == 9 and bool((y == 7.0).all())
    wy, _, ty, _ = attention(x, kc, vc, batch, 128**-0.5)
    check(w4.f16_attention(to_dev(x), cache, device_batch(w4, batch), workspace=ws), wy, ty, "in order again")


def test_wrong_arguments_are_refused(w4):
    import torch
    batch = Batch([1, 1], [30, 9], 16, seed=5)
    q, kc, vc = (to_dev(a) for a in data(batch, 16, 2, 128, 5))
    cache, kb = w4.KVCache(kc, vc), device_batch(w4, batch)
    with pytest.raises(TypeError):
        w4.f16_attention(q.float(), cache, kb)
    with pytest.raises(ValueError):
        w4.f16_attention(q.cpu(), cache, kb)
    with pytest.raises(ValueError):
        w4.f16_attention(q[:1], cache, kb)
    with pytest.raises(ValueError):
        w4.f16_attention(q[..., :64], cache, kb)
    with pytest.raises(ValueError):
        w4.f16_attention(q, cache, kb, lse=torch.empty(2, 15, device="cuda"))
    with pytest.raises(TypeError):
        w4.f16_attention(q, cache, kb, lse=torch.empty(2, 16, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        w4.f16_attention(q.transpose(1, 2).contiguous().transpose(1, 2), cache, kb)
    for kw in ({"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"scale": float("inf")}, {"window": -1}):
        with pytest.raises(w4.W4A16Error) as e:
            w4.f16_attention(q, cache, kb, **kw)
        assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_attention(q[:, :15], cache, kb)      # 15 query heads on 2
    assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_attention(q, cache, kb, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    odd = torch.empty(2, 16, 132, dtype=torch.float16, device="cuda")[..., 4:]
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_attention(odd, cache, kb)
    assert e.value.status == 3
    with pytest.raises(TypeError):
        w4.KVBatch(kb.tensors[0].long(), *kb.tensors[1:], 2, 1)
    with pytest.raises(ValueError):
        w4.KVBatch(kb.tensors[0][:1], *kb.tensors[1:], 2, 1)
    with pytest.raises(ValueError):
        w4.KVCache(kc, vc[:, :8])
    with pytest.raises(w4.W4A16Error) as e:
        w4.KVCache(kc[:, :12], vc[:, :12])          # pages of 12 tokens
    assert e.value.status == 2
