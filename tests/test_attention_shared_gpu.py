"""f16_attention beside other work on the GPU: blocks that begin late, and items joined by one block."""
import numpy as np
import pytest

from _attn import Batch
from _gpu import require_gpu, to_dev
from test_attention_gpu import data, device_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    return w4


def call_of(w4, batch, hq, hkv, d, seed):
    """(run(y, lse, stream), tokens): one call with a workspace of its own."""
    q, kc, vc = data(batch, hq, hkv, d, seed)
    tq, cache, kb = to_dev(q), w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    ws = w4.attention_workspace(cache, hq, kb.max_q_len)

    def run(y, lse=None, stream=None):
        w4.f16_attention(tq, cache, kb, y=y, lse=lse, workspace=ws, stream=stream)
    run.workspace = ws
    return run


def sentinels(n, tokens, hq, d):
    import torch
    return ([torch.full((tokens, hq, d), 7.0, dtype=torch.float16, device="cuda") for _ in range(n)],
            [torch.full((tokens, hq), 7.0, device="cuda") for _ in range(n)])


@pytest.mark.parametrize("ql,kl,hq,hkv,d", [([700], [2500], 16, 2, 128), ([2000], [2000], 8, 8, 64), ([300, 100], [2000, 1100], 16, 8, 128),
                                            ([1570], [1570], 16, 2, 128), ([90, 33], [700, 650], 28, 4, 64), ([250], [2100], 10, 2, 80)])
def test_one_block_joins_all_columns(w4, ql, kl, hq, hkv, d):
    """Items of a few parts whose columns one block joins range by range (no block may wait): the bits of the shared
    join, every time."""
    import torch
    call = call_of(w4, Batch(ql, kl, 16, seed=3), hq, hkv, d, 3)
    ys, ls = sentinels(31, sum(ql), hq, d)
    call(ys[0], ls[0])
    call.workspace.view(torch.int32)[513] = 2**30   # blocks begun in earlier calls, which the count of all calls lacks
    for y, l in zip(ys[1:], ls[1:]):
        call(y, l)
    assert w4.device_status() == 0 and not bool(call.workspace[:2048].any())
    for y, l in zip(ys[1:], ls[1:]):
        assert bool((y == ys[0]).all()) and bool((l == ls[0]).all())


@pytest.mark.parametrize("q,n,most,hq,hkv,d", [(1, 48, 8192, 16, 8, 128), (1, 48, 3000, 14, 2, 64), (24, 12, 8192, 16, 8, 128),
                                               (200, 5, 6000, 16, 2, 128), (1, 30, 4000, 8, 4, 256)])
def test_ragged_batch_beside_short_calls(w4, q, n, most, hq, hkv, d):
    """Blocks that share two items each, some beginning late as short calls of another stream hold SMs: every row is
    written, with the bits of the call alone."""
    import torch
    g = np.random.RandomState(n + d)
    kl = np.maximum(np.exp(g.uniform(np.log(most / 16), np.log(most), n)).astype(int), q)
    batch = Batch([q] * n, kl, 16, seed=n)
    big = call_of(w4, batch, hq, hkv, d, 1)
    small = call_of(w4, Batch([1], [16], 16, seed=2), 4, 1, d, 2)
    times = 40
    ys, ls = sentinels(times + 1, batch.tokens, hq, d)
    scrap = torch.empty(1, 4, d, dtype=torch.float16, device="cuda")
    big(ys[0], ls[0])
    assert w4.device_status() == 0
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(1, times + 1):
        for _ in range(4):
            small(scrap, stream=s1)
        big(ys[i], ls[i], stream=s0)
    torch.cuda.synchronize()
    assert w4.device_status() == 0
    for i in range(1, times + 1):
        assert bool((ys[i] == ys[0]).all()) and bool((ls[i] == ls[0]).all()), i
    assert not bool(big.workspace[:2048].any()) and not bool(small.workspace[:2048].any())


def test_call_on_another_stream_without_a_workspace(w4):
    """The workspace and outputs that a call makes are ordered with its stream, however busy the current one is."""
    import torch
    batch = Batch([1, 60], [9000, 3000], 16, seed=7)
    hq, hkv, d = 16, 2, 128
    q, kc, vc = data(batch, hq, hkv, d, 7)
    tq, cache, kb = to_dev(q), w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    want = w4.f16_attention(tq, cache, kb)
    rope = w4.Rope(*w4.rope_turns(d))
    want_r = w4.f16_rope(tq, rope)
    side = torch.cuda.Stream()
    # Memory that earlier work left full of ones, on both streams, for the calls to find.
    size = w4.attention_workspace_bytes(hq, hkv, d, 60)
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            full = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            del full
    torch.cuda.synchronize()
    ys = []
    for i in range(5):
        torch.cuda._sleep(4000000)   # the current stream is busy for some ms
        y = w4.f16_attention(tq, cache, kb, stream=side)
        ys.append((y, w4.f16_rope(tq, rope, stream=side)))
        scrap = torch.ones(size, dtype=torch.uint8, device="cuda")   # where a dropped workspace might have been
        del scrap
    torch.cuda.synchronize()
    assert w4.device_status() == 0
    for y, r in ys:
        assert bool((y == want).all()) and bool((r == want_r).all())


def test_windows_wider_than_32_bits(w4):
    """A window beyond any position is no window; a negative one is refused, whatever its lower 32 bits are."""
    batch = Batch([1, 40], [700, 90], 16, seed=1)
    q, kc, vc = data(batch, 4, 2, 64, 1)
    tq, cache, kb = to_dev(q), w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch)
    want = w4.f16_attention(tq, cache, kb)
    for window in (2**31 - 1, 2**31, 2**32 + 5, 2**63 - 1):
        assert bool((w4.f16_attention(tq, cache, kb, window=window) == want).all()), window
    for window in (-1, -2**31 - 1, 5 - 2**32):
        with pytest.raises(w4.W4A16Error) as e:
            w4.f16_attention(tq, cache, kb, window=window)
        assert e.value.status == 2


@pytest.mark.parametrize("hq,hkv,d,tokens", [(16, 8, 128, 60), (14, 2, 64, 9), (4, 4, 80, 100)])
def test_dominant_probability_of_few_rows(w4, hq, hkv, d, tokens):
    """Few rows over long contexts: one position far above those before it takes nearly all of a row.  Its probability
    must not lose bits of its own: bound without its rounding to binary16.

    Scores are exact (q a multiple of 1/64, k of 1/8, all columns alike): position 200 lies 2**8.. 2**15 above 128-191,
    which lie far above the rest.  Bound: the result's rounding, the other positions' roundings, exponentials and
    sums as in the oracle's."""
    g = np.random.RandomState(d)
    n = 700
    batch = Batch([tokens], [n], 16, seed=d)
    _, kc, vc = data(batch, hq, hkv, d, d, garbage=False)
    unit = 0.875 if d == 128 else 1.0 if d == 80 else 1.25
    level = np.full(n, -2.5)
    level[128:192], level[200] = 0.0, unit
    page, at = batch.slot(0, np.arange(n))
    kc[page, at] = level[:, None, None]
    steps = g.randint(45, 65, (tokens, hq)) / 64.0
    q = np.broadcast_to(steps[:, :, None], (tokens, hq, d)).astype(np.float16)
    scale = d**-0.5
    bits = steps * unit * d * scale * np.log2(np.e)
    assert 8.2 < bits.min() and bits.max() < 14.9
    y = w4.f16_attention(to_dev(np.ascontiguousarray(q)), w4.KVCache(to_dev(kc), to_dev(vc)), device_batch(w4, batch))
    assert w4.device_status() == 0
    y = y.cpu().numpy().astype(np.float64)
    p = np.exp(steps[..., None] * d * np.float64(np.float32(scale)) * (level - unit))
    p[np.broadcast_to(np.arange(n) > (n - tokens + np.arange(tokens))[:, None, None], p.shape)] = 0.0
    p /= p.sum(-1, keepdims=True)
    for h in range(hq):
        v = vc[page, at, h * hkv // hq].astype(np.float64)
        want, every = p[:, h] @ v, p[:, h] @ np.abs(v)
        rest = every - p[:, h, 200:201] * np.abs(v[200])
        tol = (2.0**-11 * (np.abs(want) + rest) + n * 2.0**-25 * np.abs(v).max()
               + (2.0**-16 + (n / 16 + 8) * 2.0**-22) * every + 2.0**-25)
        err = np.abs(y[:, h] - want)
        assert np.all(err <= tol), float((err / tol).max())
