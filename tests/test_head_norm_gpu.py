"""f16_rope and f16_kv_append with norms of the heads, against binary64."""
import numpy as np
import pytest

from _attn import TINY16, U16, Batch, rotate, rotate_tol, thetas, turns_of
from _gpu import require_gpu, to_dev

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    return w4


def weights(g, d):
    return (1.0 + 0.3 * g.standard_normal(d)).astype(np.float32)


def normed(x, w, eps=EPS):
    x = x.astype(np.float64)
    return x * w.astype(np.float64) / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))


def turned(z, pos, rot, interleaved=False):
    return rotate(z, pos, thetas(rot), 1.0, interleaved) if rot else z


def tol_of(z, pos, rot, interleaved=False):
    """rotate_tol's bound, and the norm's own fp32 arithmetic: the sum of up to 256 squares takes at most 8 + 6
    roundings on a path, the mean, eps and the square root (2 ulp) 5 more, the products 2, all of 2**-24 relative to the
    factor: below 2**-19 of each normed value that enters the result."""
    tol = (U16 + 2.0**-19) * np.abs(z) + TINY16
    if rot:
        size = np.abs(z)
        half = rot // 2
        even = np.arange(half) * 2 if interleaved else np.arange(half)
        odd = even + (1 if interleaved else half)
        pair = np.zeros_like(size)
        pair[..., even] = pair[..., odd] = size[..., even] + size[..., odd]
        tol = np.where(pair > 0, 0.0, tol) + rotate_tol(z, pos, thetas(rot), 1.0, interleaved) + 2.0**-19 * pair
    return tol


def close(got, want, tol):
    got = got.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / tol).max())


LAYOUTS = [(1, 8, 8), (16, 128, 128), (14, 64, 64), (3, 80, 40), (5, 96, 24), (7, 128, 64), (2, 256, 256), (33, 72, 8),
           (9, 136, 0), (1, 200, 16), (70, 16, 16), (4, 24, 0), (6, 248, 248)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,d,rot", LAYOUTS)
def test_rope_norm_layouts(w4, heads, d, rot, interleaved):
    g = np.random.RandomState(d + heads)
    w = weights(g, d)
    norm = w4.HeadNorm(to_dev(w), EPS)
    rope = w4.Rope(to_dev(turns_of(thetas(rot))), interleaved=interleaved) if rot else None
    for tokens in (1, 5, 131, 1700):
        x = (g.standard_normal((tokens, heads, d)) * 2.0 ** g.randint(-6, 7, (1, heads, 1))).astype(np.float16)
        pos = g.randint(0, 5000, tokens).astype(np.int32)
        y = w4.f16_rope(to_dev(x), rope, to_dev(pos), norm=norm)
        z = normed(x, w)
        close(y, turned(z, pos, rot, interleaved), tol_of(z, pos, rot, interleaved))


def test_rope_norm_extremes(w4):
    """Heads of zeros, of the smallest and of the largest values; a head that is not finite leaves the others alone."""
    import torch
    g = np.random.RandomState(0)
    w = weights(g, 128)
    norm, rope = w4.HeadNorm(to_dev(w), EPS), w4.Rope(to_dev(turns_of(thetas(128))))
    x = g.standard_normal((9, 6, 128)).astype(np.float16)
    x[:, 1] = 0.0
    x[:, 2] = 2.0**-24
    x[:, 3] = np.where(x[:, 3] > 0, 65504, -65504)
    pos = np.arange(9).astype(np.int32)
    z = normed(x, w)
    close(w4.f16_rope(to_dev(x), rope, norm=norm), turned(z, pos, 128), tol_of(z, pos, 128))
    x[:, 5, 3] = np.inf
    x[3, 4, 9] = np.nan
    y = w4.f16_rope(to_dev(x), rope, norm=norm)
    keep = np.ones((9, 6), bool)
    keep[:, 5] = keep[3, 4] = False
    close(y[torch.from_numpy(keep).cuda()], turned(z, pos, 128)[keep], tol_of(z, pos, 128)[keep])
    assert bool(y[3, 4].isnan().all()) and bool(y[:, 5].isnan().any())
    # a large eps, and none
    x = g.standard_normal((9, 6, 128)).astype(np.float16)
    for eps in (3.0, 0.0):
        z = normed(x, w, eps)
        close(w4.f16_rope(to_dev(x), rope, norm=w4.HeadNorm(to_dev(w), eps)), turned(z, pos, 128), tol_of(z, pos, 128))


def test_rope_norm_views_in_place(w4):
    import torch
    g = np.random.RandomState(1)
    w = weights(g, 64)
    x = g.standard_normal((300, 6, 64)).astype(np.float16)
    wide = torch.full((300, 8, 80), 3.0, dtype=torch.float16, device="cuda")
    part = wide[:, 1:7, 8:72]
    part.copy_(to_dev(x))
    y = w4.f16_rope(part, w4.Rope(to_dev(turns_of(thetas(64)))), norm=w4.HeadNorm(to_dev(w).half()), y=part)
    pos = np.arange(300)
    z = normed(x, w.astype(np.float16))
    close(y, turned(z, pos, 64), tol_of(z, pos, 64))
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:, 1:7, 8:72] = False
    assert bool((wide[rest] == 3.0).all())


@pytest.mark.parametrize("hq,hkv,d,rot", [(16, 8, 128, 128), (14, 2, 64, 64), (6, 3, 80, 40), (4, 1, 256, 128), (20, 1, 136, 0),
                                          (1, 1, 8, 8), (5, 5, 24, 24)])
@pytest.mark.parametrize("which", ["both", "q", "k"])
def test_append_norms(w4, hq, hkv, d, rot, which):
    """One packed projection; values and the norms that are not given are left out; unused slots stay."""
    import torch
    for ql, kl in (([1, 4, 1, 0], [0, 30, 7, 5]), ([90, 1, 260], [100, 60, 300]), ([1100, 700], [1100, 777])):
        batch = Batch(ql, kl, 16, seed=d + len(ql), extra_rows=1)
        g = np.random.RandomState(d)
        qkv = g.standard_normal((batch.tokens, hq + 2 * hkv, d)).astype(np.float16) * np.float16(3.0)
        wq, wk = weights(g, d), weights(g, d)
        t = to_dev(qkv)
        kc, vc = (torch.full((batch.pages, 16, hkv, d), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        kb = w4.KVBatch(to_dev(batch.table), to_dev(batch.offsets), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens,
                        max(ql))
        y = torch.full((batch.tokens, hq, d), 5.0, dtype=torch.float16, device="cuda")
        rope = w4.Rope(to_dev(turns_of(thetas(rot)))) if rot else None
        w4.f16_kv_append(t[:, hq:hq + hkv], t[:, hq + hkv:], w4.KVCache(kc, vc), kb, rope=rope, q=t[:, :hq], y=y,
                         q_norm=w4.HeadNorm(to_dev(wq)) if which != "k" else None,
                         k_norm=w4.HeadNorm(to_dev(wk)) if which != "q" else None)
        assert w4.device_status() == 0
        free = ~batch.used()
        for b in range(len(ql)):
            rows, pos = slice(batch.offsets[b], batch.offsets[b + 1]), batch.positions(b)
            zq = normed(qkv[rows, :hq], wq) if which != "k" else qkv[rows, :hq].astype(np.float64)
            zk = normed(qkv[rows, hq:hq + hkv], wk) if which != "q" else qkv[rows, hq:hq + hkv].astype(np.float64)
            close(y[rows], turned(zq, pos, rot), tol_of(zq, pos, rot))
            at = pos >= 0
            page, slot = batch.slot(b, pos[at])
            close(kc[page, slot], turned(zk, pos, rot)[at], tol_of(zk, pos, rot)[at])
            assert np.array_equal(vc[page, slot].cpu().numpy(), qkv[rows, hq + hkv:][at])
            old = np.arange(max(0, batch.kv_lens[b] - batch.q_lens[b]))
            page, slot = batch.slot(b, old)
            free[page, slot] = True
        assert bool((y[batch.offsets[-1]:] == 5.0).all())
        free = torch.from_numpy(free).cuda()
        assert bool((kc[free] == 7.0).all()) and bool((vc[free] == 7.0).all())


def test_calls_without_a_norm(w4):
    g = np.random.RandomState(3)
    x = g.standard_normal((200, 5, 128)).astype(np.float16)
    pos = g.randint(0, 9999, 200).astype(np.int32)
    y = w4.f16_rope(to_dev(x), w4.Rope(to_dev(turns_of(thetas(64)))), to_dev(pos))
    close(y, rotate(x, pos, thetas(64)), rotate_tol(x, pos, thetas(64)))


def test_captured_and_on_another_stream(w4):
    import torch
    g = np.random.RandomState(4)
    w = weights(g, 64)
    norm, rope = w4.HeadNorm(to_dev(w)), w4.Rope(to_dev(turns_of(thetas(64))))
    x = to_dev(g.standard_normal((40, 4, 64)).astype(np.float16))
    want = w4.f16_rope(x, rope, norm=norm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = w4.f16_rope(x, rope, norm=norm, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.f16_rope(x, rope, norm=norm, y=out)
    x.copy_(-x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


def test_wrong_norms_are_refused(w4):
    import torch
    x = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        w4.f16_rope(x, None, norm=w4.HeadNorm(w[:32]))
    with pytest.raises(ValueError):
        w4.HeadNorm(w.cpu())
    with pytest.raises(TypeError):
        w4.HeadNorm(w.double())
    with pytest.raises(ValueError):
        w4.HeadNorm(w.view(8, 8))
    page = torch.zeros(2, 16, 4, 64, dtype=torch.float16, device="cuda")
    ints = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):  # a norm of queries that are not there
        w4.f16_kv_append(x, x, w4.KVCache(page, page.clone()), w4.KVBatch(ints[:1].view(1, 1), ints, ints[:1], 3, 3),
                         q_norm=w4.HeadNorm(w))
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(w4.W4A16Error) as e:
            w4.f16_rope(x, None, norm=w4.HeadNorm(w, eps))
        assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_rope(x, None)
    assert e.value.status == 1
