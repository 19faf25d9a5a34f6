"""The attention calls refuse bad arguments on the host with the documented
codes (no CUDA call is made on these paths), and their workspace sizes follow
from their arguments alone."""
import ctypes

import pytest

from test_abi import FAKE, _status_codes, lib  # noqa: F401  (lib: the library fixture)

P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class Batch(ctypes.Structure):
    _fields_ = [("block_table", P), ("q_offsets", P), ("kv_lens", P), ("batch", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("max_q_len", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_strides", L * 3), ("v_strides", L * 3), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("box_rows", ctypes.c_int32), ("reserved", ctypes.c_int32), ("k_map", ctypes.c_uint64 * 16),
                ("v_map", ctypes.c_uint64 * 16), ("k_wide", ctypes.c_uint64 * 16), ("v_wide", ctypes.c_uint64 * 16)]


class Rotation(ctypes.Structure):
    _fields_ = [("turns", P), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("factor", F)]


def batch(**kw):
    b = Batch(FAKE, FAKE, FAKE, 2, 4, 4, 5, 3)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def cache(**kw):
    c = Cache(FAKE, FAKE, (L * 3)(4096, 256, 128), (L * 3)(4096, 256, 128), 10, 16, 2, 128, 16, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rotation(**kw):
    r = Rotation(FAKE, 64, 0, 1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def ref(x):
    return None if x is None else ctypes.addressof(x)


@pytest.fixture(scope="module")
def calls(lib):  # noqa: F811
    lib.f16_kv_cache_init.argtypes = [P, P, P, P, P, I, I, I, I]
    lib.f16_rope.argtypes = [P, L, L, P, L, L, P, P, I, I, I, P]
    lib.f16_kv_append.argtypes = [P, L, L, P, L, L, P, P, P, P, P, L, L, P, L, L, I, P]
    lib.f16_attention.argtypes = [P, L, L, P, L, L, P, I, F, I, I, P, P, P, Z, P]
    lib.f16_attention_workspace_bytes.argtypes = [I, I, I, I]
    lib.f16_attention_workspace_bytes.restype = Z

    class Calls:
        code = _status_codes()
        size = staticmethod(lib.f16_attention_workspace_bytes)
        init = staticmethod(lib.f16_kv_cache_init)

        @staticmethod
        def rope(x=FAKE, strides=(256, 128, 256, 128), y=FAKE, positions=None, r=None, tokens=3, heads=2, d=128, **kw):
            r = rotation(**kw) if r is None else r
            return lib.f16_rope(x, strides[0], strides[1], y, strides[2], strides[3], positions, ref(r) if r else None,
                                tokens, heads, d, None)

        @staticmethod
        def append(k=FAKE, v=FAKE, c=None, b=None, r=None, positions=None, q=FAKE, y=FAKE, heads=16, stride=256):
            c, b = cache() if c is None else c, batch() if b is None else b
            return lib.f16_kv_append(k, stride, 128, v, 256, 128, ref(c) if c else None, ref(b) if b else None, ref(r),
                                     positions, q, 2048, 128, y, 2048, 128, heads, None)

        @staticmethod
        def attention(q=FAKE, y=FAKE, lse=None, heads=16, scale=0.1, causal=1, window=0, c=None, b=None, ws=FAKE,
                      size=1 << 40, stride=2048):
            c, b = cache() if c is None else c, batch() if b is None else b
            return lib.f16_attention(q, stride, 128, y, 2048, 128, lse, heads, scale, causal, window,
                                     ref(c) if c else None, ref(b) if b else None, ws, size, None)

    return Calls


def test_cache_init(calls):
    c, out = calls.code, Cache()
    s = (L * 3)(4096, 256, 128)
    init = lambda o=ctypes.addressof(out), k=FAKE, v=FAKE, ks=s, vs=s, n=10, p=16, h=2, d=128: calls.init(o, k, v, ks, vs, n, p, h, d)  # noqa: E731
    for kw in ({"o": None}, {"k": None}, {"v": None}, {"ks": None}, {"vs": None}):
        assert init(**kw) == c["W4_ERR_NULL"], kw
    for kw in ({"n": 0}, {"p": 0}, {"p": 4}, {"p": 12}, {"h": 0}, {"h": 1025}, {"d": 0}, {"d": 12}, {"d": 264}):
        assert init(**kw) == c["W4_ERR_SHAPE"], kw
    for kw in ({"k": FAKE + 8}, {"v": FAKE + 2}, {"ks": (L * 3)(4096, 256, 132)}, {"vs": (L * 3)(4096, 0, 128)},
               {"ks": (L * 3)(-4096, 256, 128)}):
        assert init(**kw) == c["W4_ERR_ALIGN"], kw


def test_rope(calls):
    c = calls.code
    for kw in ({"x": None}, {"y": None}, {"turns": None}, {"r": False}):
        assert calls.rope(**kw) == c["W4_ERR_NULL"], kw
    for kw in ({"tokens": -1}, {"heads": 0}, {"heads": 1025}, {"d": 0}, {"d": 20}, {"d": 264}, {"rot": 0}, {"rot": 4},
               {"rot": 60}, {"rot": 136}, {"interleaved": 2}, {"interleaved": -1}):
        assert calls.rope(**kw) == c["W4_ERR_SHAPE"], kw
    for kw in ({"x": FAKE + 8}, {"y": FAKE + 4}, {"turns": FAKE + 4}, {"positions": FAKE + 2},
               {"strides": (260, 128, 256, 128)}, {"strides": (256, 0, 256, 128)}, {"strides": (256, 128, -256, 128)},
               {"strides": (256, 128, 256, 4)}):
        assert calls.rope(**kw) == c["W4_ERR_ALIGN"], kw
    assert calls.rope(tokens=0, x=None, y=None) == c["W4A16_OK"]


def test_batch_and_cache_checks(calls):
    c = calls.code
    for call in (calls.append, calls.attention):
        for kw in ({"block_table": None}, {"q_offsets": None}, {"kv_lens": None}):
            assert call(b=batch(**kw)) == c["W4_ERR_NULL"], kw
        assert call(b=False) == call(c=False) == call(c=cache(k=None)) == call(c=cache(v=None)) == c["W4_ERR_NULL"]
        for kw in ({"batch": 0}, {"max_pages": 0}, {"table_stride": 3}, {"total_q": -1}, {"max_q_len": -1}):
            assert call(b=batch(**kw)) == c["W4_ERR_SHAPE"], kw
        for kw in ({"num_pages": 0}, {"page_size": 12}, {"heads": 0}, {"head_dim": 260}, {"box_rows": 0},
                   {"box_rows": 64}):   # box_rows: a cache that f16_kv_cache_init did not fill in
            assert call(c=cache(**kw)) == c["W4_ERR_SHAPE"], kw
        for kw in ({"block_table": FAKE + 2}, {"q_offsets": FAKE + 1}, {"kv_lens": FAKE + 2}):
            assert call(b=batch(**kw)) == c["W4_ERR_ALIGN"], kw
        assert call(b=batch(total_q=0)) == c["W4A16_OK"]


def test_append(calls):
    c = calls.code
    for kw in ({"k": None}, {"v": None}, {"y": None}, {"r": rotation(turns=None)}):
        assert calls.append(**kw) == c["W4_ERR_NULL"], kw
    for kw in ({"heads": 0}, {"heads": 1025}, {"r": rotation(rot=136)}, {"r": rotation(rot=12)}):
        assert calls.append(**kw) == c["W4_ERR_SHAPE"], kw
    for kw in ({"k": FAKE + 8}, {"v": FAKE + 8}, {"q": FAKE + 8}, {"y": FAKE + 8}, {"positions": FAKE + 1}, {"stride": 4},
               {"stride": -256}):
        assert calls.append(**kw) == c["W4_ERR_ALIGN"], kw


def test_attention(calls):
    c = calls.code
    for kw in ({"q": None}, {"y": None}):
        assert calls.attention(**kw) == c["W4_ERR_NULL"], kw
    for kw in ({"heads": 0}, {"heads": 1}, {"heads": 15}, {"heads": 2050}, {"scale": 0.0}, {"scale": -1.0},
               {"scale": float("nan")}, {"scale": float("inf")}, {"causal": 2}, {"causal": -1}, {"window": -1},
               {"b": batch(total_q=2**30), "heads": 32}):
        assert calls.attention(**kw) == c["W4_ERR_SHAPE"], kw
    for kw in ({"q": FAKE + 8}, {"y": FAKE + 8}, {"ws": FAKE + 8}, {"lse": FAKE + 2}, {"stride": 2052}):
        assert calls.attention(**kw) == c["W4_ERR_ALIGN"], kw
    assert calls.attention(ws=None) == c["W4_ERR_WORKSPACE"]
    assert calls.attention(size=calls.size(16, 2, 128, 3) - 1) == c["W4_ERR_WORKSPACE"]


def test_workspace_sizes(calls):
    assert calls.size(16, 2, 128, 1) > 0
    for bad in ((15, 2, 128, 1), (0, 1, 128, 1), (2, 0, 128, 1), (2, 1, 12, 1), (2, 1, 264, 1), (2, 1, 128, -1)):
        assert calls.size(*bad) == 0, bad
    for d in (8, 64, 128, 256):   # more tokens of a sequence never need less
        sizes = [calls.size(16, 2, d, n) for n in (0, 1, 2, 4, 16, 100, 10**4)]
        assert sizes == sorted(sizes) and sizes[-1] < 1 << 28
