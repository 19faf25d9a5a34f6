"""f16_lora against binary64."""
import numpy as np
import pytest

from _attn import TINY16, U16
from _gpu import require_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    yield w4
    assert w4.device_status() == 0


class Case:
    """Seeded adapters, rows and the result in binary64 with a bound on |gpu - oracle|:

    h = x A^T in fp32: at most K / 16 + 24 additions of 2**-23 relative to sum |x a|
    h as hi + lo:      2**-21 of the row's largest
    the second sum:    rank / 8 + 4 additions of 2**-23 relative to sum |h b|
    scale, the power of two, y + delta: 2**-22 of |delta| + |y|
    the rounding:      U16 |out| + TINY16
    """

    def __init__(self, m, k, columns, rank, adapters, ids, seed=0, with_scale=True, big=1.0):
        g = np.random.RandomState(seed)
        self.ids, self.columns = np.asarray(ids, np.int32), columns
        n, s = sum(columns), len(columns)
        self.x = g.standard_normal((m, k)).astype(np.float16)
        self.y = g.standard_normal((m, n)).astype(np.float16)
        self.a = (big * g.standard_normal((adapters, s, rank, k)) / np.sqrt(k)).astype(np.float16)
        self.b = (g.standard_normal((adapters, n, rank)) * 0.1).astype(np.float16)
        self.scale = (2.0 * g.random_sample(adapters) - 0.5).astype(np.float32) if with_scale else None

    def want(self):
        out, tol = self.y.astype(np.float64), np.zeros(self.y.shape)
        edges = np.cumsum([0, *self.columns])
        k, rank = self.x.shape[1], self.b.shape[2]
        for m, i in enumerate(self.ids):
            if not 0 <= i < len(self.a):
                continue
            sc = 1.0 if self.scale is None else float(self.scale[i])
            x = self.x[m].astype(np.float64)
            hs = [self.a[i, s].astype(np.float64) @ x * sc for s in range(len(self.columns))]
            es = [(k / 16 + 24) * 2.0**-23 * (np.abs(self.a[i, s].astype(np.float64)) @ np.abs(x)) * abs(sc)
                  for s in range(len(self.columns))]
            top = max(np.abs(h).max() for h in hs)
            for s, h in enumerate(hs):
                c = slice(edges[s], edges[s + 1])
                b = self.b[i, c].astype(np.float64)
                out[m, c] += b @ h
                tol[m, c] = (np.abs(b) @ (es[s] + 2.0**-21 * top + (rank / 8 + 4) * 2.0**-23 * np.abs(h))
                             + 2.0**-22 * (np.abs(b @ h) + np.abs(self.y[m, c])))
        return out, tol + U16 * np.abs(out) + TINY16

    def adapters(self, w4):
        return w4.Adapters(to_dev(self.a), to_dev(self.b), None if self.scale is None else to_dev(self.scale),
                           columns=self.columns)

    def check(self, w4, got, want=None):
        out, tol = want or self.want()
        got = got.cpu().numpy()
        err = np.abs(got.astype(np.float64) - out)
        assert np.all(err <= tol), float(np.nanmax(err / tol))
        none = (self.ids < 0) | (self.ids >= len(self.a))
        assert np.array_equal(got[none].view(np.uint16), self.y[none].view(np.uint16))


def run(w4, c, in_place=False):
    import torch
    y = to_dev(c.y)
    out = y if in_place else torch.full_like(y, 7.0)
    got = w4.f16_lora(to_dev(c.x), c.adapters(w4), to_dev(c.ids), y, out=None if in_place else out)
    assert got is out or in_place and got is y
    if not in_place:
        assert np.array_equal(y.cpu().numpy(), c.y)
    return got


def some_ids(m, adapters, seed, none=0.2):
    g = np.random.RandomState(seed)
    ids = g.randint(0, adapters, m)
    ids[g.random_sample(m) < none] = -1
    return ids


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("k,columns", [(8, (8,)), (64, (40,)), (256, (136, 8)), (200, (32, 8, 72)), (896, (896, 128, 128)),
                                       (1024, (8, 16, 24, 32))])
def test_ranks_and_slices(w4, rank, k, columns):
    for m in (1, 5, 17, 40, 70):
        c = Case(m, k, columns, rank, 5, some_ids(m, 5, m), seed=rank + m)
        c.check(w4, run(w4, c, in_place=m % 2 == 0))


@pytest.mark.parametrize("m", [1, 2, 8, 16, 33, 64, 100, 300, 1024, 1025, 2100])
@pytest.mark.parametrize("pattern", ["one", "all", "many", "runs", "none"])
def test_mixes_of_rows(w4, m, pattern):
    adapters = 12
    ids = {"one": np.full(m, 7), "all": np.arange(m) % adapters, "many": some_ids(m, adapters, m, 0.5),
           "runs": np.sort(some_ids(m, adapters, m))[::-1].copy(), "none": np.full(m, -3)}[pattern]
    c = Case(m, 136, (200, 56), 16, adapters, ids, seed=m)
    want = c.want()
    first = run(w4, c)
    c.check(w4, first, want)
    again = run(w4, c, in_place=True)
    assert np.array_equal(first.cpu().numpy(), again.cpu().numpy())


@pytest.mark.parametrize("k,columns,rank,m", [(2048, (2048, 256, 256), 16, 9), (2048, (11008, 11008), 32, 3),
                                              (11008, (2048,), 64, 20), (2048, (2048, 256, 256), 128, 130),
                                              (2048, (1000,), 64, 700)])
def test_projection_sizes(w4, k, columns, rank, m):
    c = Case(m, k, columns, rank, 4, some_ids(m, 4, rank), seed=m)
    c.check(w4, run(w4, c))


@pytest.mark.parametrize("rank,slices", [(32, 3), (128, 3), (128, 4), (24, 4), (64, 3), (72, 4)])
@pytest.mark.parametrize("k,m", [(2048, 300), (2056, 1100), (5000, 150)])
@pytest.mark.parametrize("order", ["runs", "mixed"])
def test_rings_of_long_rows(w4, rank, slices, k, m, order):
    """Items of more than 16 rows whose K passes the ring several times: rows that lie in a row and gathered ones, all
    ranks from 96 to 512 (items of 64 rows above 192, two boxes of A above 256), a K that ends inside a stage."""
    columns = (72, 40, 8, 16)[:slices]
    ids = np.repeat([2, -1, 0, 1], [m // 2, m // 10, m // 4, m - m // 2 - m // 10 - m // 4])
    if order == "mixed":
        ids = np.random.RandomState(m).permutation(ids)
    c = Case(m, k, columns, rank, 3, ids, seed=rank + m)
    c.check(w4, run(w4, c, in_place=order == "mixed"))


def test_many_adapters(w4):
    """Histograms of more buckets than threads, and the most there can be."""
    for adapters, m in ((300, 257), (4096, 600)):
        c = Case(m, 64, (48,), 8, adapters, some_ids(m, adapters, m, 0.05), seed=adapters, with_scale=False)
        c.ids[0], c.ids[1] = adapters - 1, 0
        c.check(w4, run(w4, c))


def test_large_and_small_values(w4):
    """x A^T beyond binary16's range and far below it, and scales of both kinds."""
    for big in (30.0, 2.0**-10):
        c = Case(40, 512, (64, 32), 16, 3, some_ids(40, 3, 1), seed=5, big=big)
        if big > 1:
            c.x = (c.x * np.float16(300)).astype(np.float16)
            c.b = (c.b.astype(np.float64) * 1e-4).astype(np.float16)
        c.scale = np.array([1000.0, 1e-6, -3.0], np.float32)
        c.check(w4, run(w4, c))
    c = Case(4, 64, (64,), 16, 3, [0, 1, 2, 0], seed=6)
    c.scale = np.array([0.0, 1.0, 0.0], np.float32)
    c.x[1] = 0
    assert np.array_equal(run(w4, c).cpu().numpy(), c.y)


def test_rows_that_are_not_finite_stay_apart(w4):
    m = 50
    c = Case(m, 128, (64, 40), 24, 4, np.arange(m) % 4, seed=7)
    want = c.want()
    c.x[6, 3], c.x[9, 100] = np.inf, np.nan          # adapters 2 and 1
    c.y[20, 5] = np.inf
    c.a[3, 0, 2, 9] = np.nan                         # an adapter of its own rows only
    got = run(w4, c).cpu().numpy()
    bad = np.zeros(m, bool)
    bad[[6, 9]] = True
    bad[3::4] = True
    err = np.abs(got[~bad].astype(np.float64) - want[0][~bad])
    ok = err <= want[1][~bad]
    ok[np.flatnonzero(~bad) == 20, 5] = True
    assert np.all(ok) and np.isposinf(got[20, 5])
    assert not np.isfinite(got[6]).any() and np.isnan(got[9]).all() and np.isnan(got[3, :64]).all()


@pytest.mark.parametrize("m,rank", [(9, 16), (40, 16), (40, 40), (300, 72)])
def test_a_slice_that_is_not_finite_leaves_the_others(w4, m, rank):
    """An adapter with an infinity or a NaN in one slice's A: the columns of its other slices are as without it, with
    x A^T beyond binary16's range as well as below it."""
    for size in (30.0, 2.0**-12):
        c = Case(m, 128, (64, 40, 8), rank, 3, np.arange(m) % 3, seed=13, big=size)
        c.x = (c.x * np.float16(300 if size > 1 else 1)).astype(np.float16)
        c.b = (c.b.astype(np.float64) * (1e-6 if size > 1 else 1.0)).astype(np.float16)
        c.scale = np.array([1000.0, 1.0, 1e-3] if size > 1 else [1.0, 1e-3, 0.1], np.float32)
        for value in (np.inf, np.nan):
            c.a[:, 0, 3, 5] = 0
            out, tol = c.want()
            c.a[:, 0, 3, 5] = value
            got = run(w4, c, in_place=value == np.inf).cpu().numpy()
            assert np.all(np.abs(got[:, 64:].astype(np.float64) - out[:, 64:]) <= tol[:, 64:])
            assert not np.isfinite(got[:, :64][np.abs(c.x[:, 5]) > 0]).all(axis=1).any()


def test_strides(w4):
    """Rows of x, y and out inside wider tensors, adapters apart from each other; nothing else is written."""
    import torch
    c = Case(30, 64, (40, 24), 16, 3, some_ids(30, 3, 2), seed=8)
    n = 64
    x = torch.zeros(30, 96, dtype=torch.float16, device="cuda")
    x[:, 16:80] = to_dev(c.x)
    y = torch.full((30, 200), 3.0, dtype=torch.float16, device="cuda")
    y[:, 8:8 + n] = to_dev(c.y)
    out = torch.full((30, 80), 5.0, dtype=torch.float16, device="cuda")
    a = torch.zeros(3, 3, 2, 16, 64, dtype=torch.float16, device="cuda")
    a[:, 1] = to_dev(c.a)
    b = torch.zeros(3, 2, n, 16, dtype=torch.float16, device="cuda")
    b[:, 0] = to_dev(c.b)
    ad = w4.Adapters(a[:, 1], b[:, 0], to_dev(c.scale), columns=c.columns)
    w4.f16_lora(x[:, 16:80], ad, to_dev(c.ids), y[:, 8:8 + n], out=out[:, 16:80])
    c.check(w4, out[:, 16:80])
    assert bool((out[:, :16] == 5.0).all()) and bool((y[:, 8 + n:] == 3.0).all()) and bool((y[:, :8] == 3.0).all())
    w4.f16_lora(x[:, 16:80], ad, to_dev(c.ids), y[:, 8:8 + n])
    c.check(w4, y[:, 8:8 + n])
    assert bool((y[:, 8 + n:] == 3.0).all()) and bool((y[:, :8] == 3.0).all())


def test_far_rows_and_adapters(w4):
    """Rows of out and an adapter beyond 2**32 elements."""
    import torch
    if torch.cuda.mem_get_info()[0] < 3 * 2**34:
        pytest.skip("not enough device memory")
    c = Case(9, 64, (64,), 16, 2, [0, 1, 1, 0, -1, 1, 0, 0, 1], seed=9)
    far = torch.empty(9, 2**29 + 64, dtype=torch.float16, device="cuda")
    out = far[:, 2**29:]
    apart = 2**32 + 1024
    store = torch.empty(apart + 4096, dtype=torch.float16, device="cuda")
    a = store.as_strided((2, 1, 16, 64), (apart, 1024, 64, 1))
    a.copy_(to_dev(c.a))
    w4.f16_lora(to_dev(c.x), w4.Adapters(a, to_dev(c.b), to_dev(c.scale)), to_dev(c.ids), to_dev(c.y), out=out)
    c.check(w4, out.contiguous())
    del far, out, store, a
    torch.cuda.empty_cache()


def test_bad_ids_count_as_none_and_are_reported(w4):
    c = Case(20, 64, (64,), 16, 3, some_ids(20, 3, 4), seed=10)
    c.ids[[2, 11]] = 3, 2**31 - 1
    c.ids[3] = -(2**31)
    c.check(w4, run(w4, c))
    assert w4.device_status() == 9 and w4.device_status() == 0


def test_captured_streams_and_two_at_once(w4):
    import torch
    c = Case(70, 256, (128, 64), 16, 6, some_ids(70, 6, 5), seed=11)
    ad, x, y, ids = c.adapters(w4), to_dev(c.x), to_dev(c.y), to_dev(c.ids)
    out = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.f16_lora(x, ad, ids, y, out=out)
    graph.replay()
    torch.cuda.synchronize()
    c.check(w4, out)
    c.ids = some_ids(70, 6, 77).astype(np.int32)
    ids.copy_(to_dev(c.ids))
    graph.replay()
    torch.cuda.synchronize()
    want = c.want()
    c.check(w4, out, want)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros_like(y) for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, o in zip(side, outs):
            w4.f16_lora(x, ad, ids, y, out=o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out)
    empty = w4.f16_lora(x[:0], ad, ids[:0], y[:0])
    assert empty.shape == (0, 192)


def test_one_workspace_for_fewer_rows(w4):
    """A workspace for many rows, with garbage in it, serves calls with fewer, one after the other."""
    ws = w4.lora_workspace(Case(1, 64, (256, 256), 48, 3, [0]).adapters(w4), 1500)
    ws.fill_(0xFF)
    for m in (1500, 1, 17, 33, 200, 1025):
        c = Case(m, 64, (256, 256), 48, 3, some_ids(m, 3, m), seed=m)
        y = to_dev(c.y)
        w4.f16_lora(to_dev(c.x), c.adapters(w4), to_dev(c.ids), y, workspace=ws)
        c.check(w4, y)


def test_wrong_arguments_are_refused(w4):
    import torch
    c = Case(4, 64, (40, 24), 16, 3, [0, 1, 2, -1], seed=12)
    ad, x, y, ids = c.adapters(w4), to_dev(c.x), to_dev(c.y), to_dev(c.ids)
    a, b = to_dev(c.a), to_dev(c.b)
    with pytest.raises(ValueError):
        w4.Adapters(a, b)                       # two slices, one width
    with pytest.raises(ValueError):
        w4.Adapters(a, b, columns=(40, 32))
    with pytest.raises(ValueError):
        w4.Adapters(a, b[:2], columns=(40, 24))
    with pytest.raises(TypeError):
        w4.Adapters(a.float(), b, columns=(40, 24))
    with pytest.raises(ValueError):
        w4.Adapters(a, b, scale=torch.ones(2, device="cuda"), columns=(40, 24))
    with pytest.raises(ValueError):
        w4.f16_lora(x[:, :56], ad, ids, y)
    with pytest.raises(ValueError):
        w4.f16_lora(x, ad, ids[:3], y)
    with pytest.raises(TypeError):
        w4.f16_lora(x, ad, ids.long(), y)
    with pytest.raises(TypeError):
        w4.f16_lora(x, ad, ids, y.float())
    with pytest.raises(ValueError):
        w4.f16_lora(x, ad, ids, y, out=y[:, :56])
    for columns in ((36, 28), (44, 20)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.f16_lora(x, w4.Adapters(a, b, columns=columns), ids, y)
        assert e.value.status == 2
    with pytest.raises(w4.W4A16Error) as e:    # rank 136
        w4.f16_lora(x, w4.Adapters(torch.zeros(1, 136, 64, dtype=torch.float16, device="cuda"),
                                   torch.zeros(1, 64, 136, dtype=torch.float16, device="cuda")), ids, y)
    assert e.value.status == 2
    wide = torch.zeros(4, 68, dtype=torch.float16, device="cuda")
    with pytest.raises(w4.W4A16Error) as e:
        w4.f16_lora(wide[:, :64], ad, ids, y)
    assert e.value.status == 3
