"""f16_rope and f16_kv_append against the binary64 oracle."""
import numpy as np
import pytest

from _attn import Batch, rotate, rotate_tol, thetas, turns_of
from _gpu import require_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    return w4


def rope_of(w4, theta, factor=1.0, interleaved=False):
    return w4.Rope(to_dev(turns_of(theta)), factor=factor, interleaved=interleaved)


def close(got, want, tol, what="y"):
    got = got.cpu().numpy().astype(np.float64)
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, float((err / tol).max()))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,d,rot", [(1, 8, 8), (16, 128, 128), (14, 64, 64), (3, 80, 32), (5, 96, 24), (7, 128, 64),
                                         (2, 256, 256), (33, 72, 8), (9, 136, 136), (1, 200, 16), (70, 16, 16)])
def test_rope_layouts(w4, heads, d, rot, interleaved):
    g = np.random.RandomState(d + rot)
    for tokens in (1, 5, 130):
        x = g.standard_normal((tokens, heads, d)).astype(np.float16)
        pos = g.randint(0, 5000, tokens).astype(np.int32)
        y = w4.f16_rope(to_dev(x), rope_of(w4, thetas(rot), 1.25, interleaved), to_dev(pos))
        close(y, rotate(x, pos, thetas(rot), 1.25, interleaved), rotate_tol(x, pos, thetas(rot), 1.25, interleaved))
        tail = y[..., rot:].cpu().numpy()
        assert np.array_equal(tail, x[..., rot:])


@pytest.mark.parametrize("tokens,heads,d,rot", [(700, 16, 128, 128), (1501, 16, 128, 64), (2600, 9, 136, 136), (3001, 11, 80, 32),
                                                (5000, 33, 72, 8), (6000, 1, 64, 64), (2500, 35, 256, 256)])
def test_rope_many_tokens(w4, tokens, heads, d, rot):
    """One, four and eight heads to a lane, and groups of heads that are not full."""
    g = np.random.RandomState(tokens)
    x = g.standard_normal((tokens, heads, d)).astype(np.float16)
    pos = g.randint(0, 100000, tokens).astype(np.int32)
    y = w4.f16_rope(to_dev(x), rope_of(w4, thetas(rot), 1.0), to_dev(pos))
    close(y, rotate(x, pos, thetas(rot)), rotate_tol(x, pos, thetas(rot)))


def test_rope_far_and_negative_positions(w4):
    """The angle's reduction is exact at every int32 position; a negative one turns back."""
    pos = np.array([0, 1, -1, 131071, 10**6, 2**24 + 1, 2**31 - 1, -2**31, -12345], np.int32)
    g = np.random.RandomState(0)
    x = g.standard_normal((len(pos), 4, 128)).astype(np.float16)
    turns = turns_of(thetas(128, 1e6))
    frac = (pos.astype(np.int64)[:, None] * turns[None]).astype(np.float64) * 2.0**-64 * 2 * np.pi  # reduced exactly
    rope = w4.Rope(to_dev(turns))
    y = w4.f16_rope(to_dev(x), rope, to_dev(pos))
    z = (x[..., :64].astype(np.float64) + 1j * x[..., 64:]) * np.exp(1j * frac)[:, None, :]
    want = np.concatenate([z.real, z.imag], -1)
    size = np.abs(x[..., :64].astype(np.float64)) + np.abs(x[..., 64:])
    tol = 2.0**-11 * np.abs(want) + 2.0**-20 * np.concatenate([size, size], -1) + 2.0**-25
    close(y, want, tol)
    back = w4.f16_rope(y, rope, to_dev((-pos.astype(np.int64)).clip(-2**31, 2**31 - 1).astype(np.int32)))
    keep = pos != -2**31
    assert np.abs(back.cpu().numpy().astype(np.float64)[keep] - x[keep]).max() <= 2.0**-9 * np.abs(x).max()


def test_rope_in_place_strided_and_without_positions(w4):
    import torch
    g = np.random.RandomState(1)
    theta = thetas(64)
    for interleaved in (False, True):
        x = g.standard_normal((300, 6, 64)).astype(np.float16)
        wide = torch.full((300, 8, 80), 3.0, dtype=torch.float16, device="cuda")
        part = wide[:, 1:7, 8:72]
        part.copy_(to_dev(x))
        w4.f16_rope(part, rope_of(w4, theta, 1.0, interleaved), y=part)
        close(part, rotate(x, np.arange(300), theta, 1.0, interleaved), rotate_tol(x, np.arange(300), theta, 1.0, interleaved))
        part.fill_(3.0)
        assert bool((wide == 3.0).all())
        hm = to_dev(x).transpose(0, 1).contiguous().transpose(0, 1)   # heads outermost
        y = w4.f16_rope(hm, rope_of(w4, theta, 1.0, interleaved))
        close(y, rotate(x, np.arange(300), theta, 1.0, interleaved), rotate_tol(x, np.arange(300), theta, 1.0, interleaved))
    assert w4.f16_rope(torch.empty(0, 6, 64, dtype=torch.float16, device="cuda"), rope_of(w4, theta)).shape == (0, 6, 64)


def test_rope_other_stream(w4):
    import torch
    x = torch.randn(4000, 16, 128, device="cuda").half()
    rope = rope_of(w4, thetas(128))
    want = w4.f16_rope(x, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = w4.f16_rope(x, rope)
    b = w4.f16_rope(x, rope, stream=side)
    side.synchronize()
    assert bool((a == want).all()) and bool((b == want).all())


def append_case(w4, batch, hq, hkv, d, rot, interleaved=False, positions=None, head_major=False, with_q=True, seed=0,
                garbage=True):
    import torch
    g = np.random.RandomState(seed)
    q = g.standard_normal((batch.tokens, hq, d)).astype(np.float16)
    k, v = (g.standard_normal((batch.tokens, hkv, d)).astype(np.float16) for _ in range(2))
    kc, vc = (g.standard_normal((batch.pages, batch.page, hkv, d)).astype(np.float16) for _ in range(2))
    tk, tv = to_dev(kc), to_dev(vc)
    if head_major:
        tk, tv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (tk, tv))
    theta = thetas(rot) if rot else np.zeros(0)
    rope = rope_of(w4, theta, 1.0, interleaved) if rot else None
    cache = w4.KVCache(tk, tv)
    kb = w4.KVBatch(to_dev(batch.table), to_dev(batch.offsets), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens,
                    int(batch.q_lens.max()))
    ty = torch.full((batch.tokens, hq, d), 9.0, dtype=torch.float16, device="cuda")
    got = w4.f16_kv_append(to_dev(k), to_dev(v), cache, kb, rope=rope, q=to_dev(q) if with_q else None,
                           y=ty if with_q else None, positions=None if positions is None else to_dev(positions))
    assert w4.device_status() == 0
    n = int(batch.offsets[-1])
    where = np.concatenate([batch.positions(b) for b in range(len(batch.q_lens))]).astype(np.int64)
    turn = where if positions is None else positions[:n].astype(np.int64)
    want_k, want_v, tol_k = kc.astype(np.float64), vc.copy(), np.zeros(kc.shape)
    rk = rotate(k[:n], turn, theta, 1.0, interleaved)
    tolk = rotate_tol(k[:n], turn, theta, 1.0, interleaved)
    for b in range(len(batch.q_lens)):
        for i, p in enumerate(batch.positions(b)):
            if p < 0:
                continue
            t = batch.offsets[b] + i
            pg, at = batch.slot(b, p)
            want_k[pg, at], want_v[pg, at], tol_k[pg, at] = rk[t], v[t], tolk[t]
    close(tk, want_k, tol_k, "k_cache")   # slots of other positions: bit for bit
    assert np.array_equal(tv.cpu().numpy().view(np.uint16), want_v.view(np.uint16))
    if with_q:
        close(got[:n], rotate(q[:n], turn, theta, 1.0, interleaved), rotate_tol(q[:n], turn, theta, 1.0, interleaved), "q")
        assert bool((ty[n:] == 9.0).all())
    else:
        assert got is None


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot", [(16, 2, 128, 128), (16, 8, 128, 64), (14, 2, 64, 64), (1, 1, 8, 8), (5, 1, 80, 32),
                                          (6, 3, 96, 96), (4, 2, 256, 128), (20, 1, 136, 136), (16, 2, 128, 0)])
def test_append_layouts(w4, hq, hkv, d, rot, interleaved):
    append_case(w4, Batch([1, 37, 4, 1], [1, 40, 133, 200], 16, seed=d), hq, hkv, d, rot, interleaved)


@pytest.mark.parametrize("page", [8, 16, 24, 64, 1000])
def test_append_pages_and_views(w4, page):
    batch = Batch([3, 0, 90, 1], [70, 55, 90, 1], page, seed=page, extra_rows=2)
    append_case(w4, batch, 16, 2, 128, 128, head_major=True)
    append_case(w4, batch, 16, 2, 128, 128, with_q=False)


def test_append_own_positions(w4):
    batch = Batch([3, 5], [30, 25], 16, seed=1, extra_rows=1)
    append_case(w4, batch, 4, 2, 64, 64, positions=np.array([9, 70000, 3, 0, -5, 2, 1, 8, 4], np.int32))


def test_append_padded_slots(w4):
    """A token at a negative position is not written; its query is rotated all the same."""
    append_case(w4, Batch([1, 1, 4, 0, 1], [0, 17, 2, 0, 0], 16, seed=2), 16, 2, 128, 128)


@pytest.mark.parametrize("n", [33, 1025, 2500])
def test_append_many_sequences(w4, n):
    g = np.random.RandomState(n)
    ql = g.randint(0, 3, n)
    append_case(w4, Batch(ql, np.maximum(ql, g.randint(0, 30, n)), 8, seed=n), 2, 1, 64, 64)


@pytest.mark.parametrize("hq,hkv,d,rot", [(16, 8, 128, 128), (14, 2, 64, 64), (5, 3, 80, 32), (20, 1, 136, 0)])
def test_append_many_tokens(w4, hq, hkv, d, rot):
    """One, four and eight heads to a lane."""
    for ql in ([60], [700, 3], [1500, 1, 900], [5000]):
        append_case(w4, Batch(ql, [n + 7 for n in ql], 16, seed=d), hq, hkv, d, rot)


def test_append_packed_projection(w4):
    """q, k and v as views of one [tokens][heads][dim] projection, the queries rotated in place."""
    import torch
    batch = Batch([2, 50], [9, 80], 16, seed=4)
    g = np.random.RandomState(4)
    x = g.standard_normal((batch.tokens, 20, 128)).astype(np.float16)
    t = to_dev(x)
    kc = torch.zeros(batch.pages, 16, 2, 128, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    kb = w4.KVBatch(to_dev(batch.table), to_dev(batch.offsets), to_dev(batch.kv_lens.astype(np.int32)), batch.tokens, 50)
    theta = thetas(128)
    w4.f16_kv_append(t[:, 16:18], t[:, 18:], w4.KVCache(kc, vc), kb, rope=rope_of(w4, theta), q=t[:, :16], y=t[:, :16])
    pos = np.concatenate([batch.positions(0), batch.positions(1)])
    close(t[:, :16], rotate(x[:, :16], pos, theta), rotate_tol(x[:, :16], pos, theta))
    assert np.array_equal(t[:, 16:].cpu().numpy(), x[:, 16:])
    pg, at = batch.slot(1, batch.positions(1))
    close(kc[pg, at], rotate(x[2:, 16:18], pos[2:], theta), rotate_tol(x[2:, 16:18], pos[2:], theta))


def test_append_far_pages(w4):
    """Pages that lie beyond 2**32 elements of the cache."""
    import torch
    page, hkv, d = 64, 2, 128
    pages = 2**32 // (page * hkv * d) + 8
    if torch.cuda.mem_get_info()[0] < 4 * 2**32 + 2**31:
        pytest.skip("not enough device memory")
    kc, vc = (torch.zeros(pages, page, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    k, v = (torch.randn(3, hkv, d, device="cuda").half() for _ in range(2))
    kb = w4.KVBatch(to_dev(np.array([[5, pages - 1]], np.int32)), to_dev(np.array([0, 3], np.int32)),
                    to_dev(np.array([66], np.int32)), 3, 3)
    w4.f16_kv_append(k, v, w4.KVCache(kc, vc), kb)
    assert bool((kc[pages - 1, :2] == k[1:]).all()) and bool((vc[pages - 1, :2] == v[1:]).all())
    assert bool((kc[5, 63] == k[0]).all()) and bool((vc[5, 63] == v[0]).all())
    del kc, vc
    torch.cuda.empty_cache()


def test_append_bad_pages_are_skipped_and_reported(w4):
    import torch
    kc, vc = (torch.zeros(4, 16, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    k, v = (torch.ones(3, 1, 64, device="cuda").half() for _ in range(2))
    cache = w4.KVCache(kc, vc)
    kb = w4.KVBatch(to_dev(np.array([[4], [-1], [2]], np.int32)), to_dev(np.array([0, 1, 2, 3], np.int32)),
                    to_dev(np.array([5, 5, 5], np.int32)), 3, 1)
    w4.f16_kv_append(k, v, cache, kb)
    assert w4.device_status() == 9 and w4.device_status() == 0
    assert int((kc != 0).sum()) == 64 and bool((kc[2, 4] == 1).all()) and int((vc != 0).sum()) == 64


def test_turns_of_scaled_contexts(w4):
    """rope_turns against the formulas, in the fraction of a turn that it holds."""
    import math
    rot, base, s, L = 128, 1e6, 4.0, 32768
    i = np.arange(64)
    th = base ** (-2.0 * i / rot)
    lo = max(math.floor(rot * math.log(L / (32 * 2 * math.pi)) / (2 * math.log(base))), 0)
    hi = min(math.ceil(rot * math.log(L / (1 * 2 * math.pi)) / (2 * math.log(base))), 63)
    r = np.clip((i - lo) / (hi - lo), 0, 1)
    mix = np.clip((L * th / (2 * np.pi) - 1) / 3, 0, 1)
    want = {None: th, "linear": th / s, "ntk": (base * s ** (rot / (rot - 2))) ** (-2.0 * i / rot),
            "yarn": th * (1 - r) + th / s * r, "bands": th * mix + th / s * (1 - mix)}
    for method, t in want.items():
        turns, factor = w4.rope_turns(rot, base, method, s, L)
        got = turns.cpu().numpy().view(np.uint64).astype(np.float64) * 2.0**-64 * 2 * np.pi
        assert np.all(np.abs(got - t) <= 1e-12 * t), method
        assert factor == (0.1 * math.log(s) + 1 if method == "yarn" else 1.0)


def test_wrong_arguments_are_refused(w4):
    import torch
    x = torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda")
    rope = rope_of(w4, thetas(64))
    with pytest.raises(TypeError):
        w4.f16_rope(x.float(), rope)
    with pytest.raises(ValueError):
        w4.f16_rope(x[0], rope)
    with pytest.raises(ValueError):
        w4.f16_rope(x, rope, y=x[:2])
    with pytest.raises(ValueError):
        w4.f16_rope(x, rope, to_dev(np.zeros(2, np.int32)))
    with pytest.raises(TypeError):
        w4.f16_rope(x, rope, to_dev(np.zeros(3, np.int64)))
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_rope(x, rope_of(w4, thetas(72)))      # more than the head
    assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_rope(x, rope_of(w4, np.ones(6)))      # rot 12
    assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_rope(torch.zeros(3, 4, 68, dtype=torch.float16, device="cuda")[..., :64], rope)   # rows of 136 bytes
    assert e.value.status == 3
    with pytest.raises(TypeError):
        w4.Rope(torch.zeros(32, device="cuda"))
    with pytest.raises(ValueError):
        w4.rope_turns(20)
    with pytest.raises(ValueError):
        w4.rope_turns(64, method="yarn", stretch=2.0)
    kc = torch.zeros(4, 16, 2, 64, dtype=torch.float16, device="cuda")
    cache = w4.KVCache(kc, kc.clone())
    kb = w4.KVBatch(to_dev(np.zeros((1, 1), np.int32)), to_dev(np.array([0, 3], np.int32)), to_dev(np.array([3], np.int32)), 3, 3)
    k = x[:, :2].contiguous()
    with pytest.raises(ValueError):
        w4.f16_kv_append(x, x, cache, kb)             # 4 heads into 2
    with pytest.raises(ValueError):
        w4.f16_kv_append(k[:2], k[:2], cache, kb)
    with pytest.raises(ValueError):
        w4.f16_kv_append(k, k, cache, kb, y=x)
    with pytest.raises(ValueError):
        w4.f16_kv_append(k, k, cache, kb, q=x[..., :32])
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_kv_append(k, k, cache, kb, rope=rope_of(w4, thetas(128)))
    assert e.value.status == 2


@pytest.mark.parametrize("tokens", [1, 30])
def test_append_skips_sequences_out_of_range(w4, tokens):
    """A length past the table or below zero, or offsets past the tensors: reported, and the cached tokens stay."""
    import torch
    g = np.random.RandomState(tokens)
    n, page, pages = 3, 16, 4
    table = np.arange(n * pages).reshape(n, pages).astype(np.int32)
    kc, vc = (to_dev(g.standard_normal((n * pages, page, 2, 64)).astype(np.float16)) for _ in range(2))
    k, v = (to_dev(g.standard_normal((n * tokens, 2, 64)).astype(np.float16)) for _ in range(2))
    good = np.array([40, 50, 60], np.int32)
    offsets = (np.arange(n + 1) * tokens).astype(np.int32)
    past = offsets.copy()
    past[-1] += 5
    for lens, offs, bad in ((np.array([40, 65, 60], np.int32), offsets, 1), (np.array([40, 2**31 - 1, 60], np.int32), offsets, 1),
                            (np.array([-1, 50, 60], np.int32), offsets, 0), (good, past, 2)):
        a, b = kc.clone(), vc.clone()
        kb = w4.KVBatch(to_dev(table), to_dev(offs), to_dev(lens), n * tokens, tokens)
        w4.f16_kv_append(k, v, w4.KVCache(a, b), kb)
        assert w4.device_status() == 9 and w4.device_status() == 0
        want_k, want_v = kc.clone(), vc.clone()
        for s in range(n):
            for i in range(tokens):
                p = int(good[s]) - tokens + i
                if s != bad:
                    want_k[s * pages + p // page, p % page] = k[s * tokens + i]
                    want_v[s * pages + p // page, p % page] = v[s * tokens + i]
        assert bool((a == want_k).all()) and bool((b == want_v).all()), (lens.tolist(), offs.tolist())
