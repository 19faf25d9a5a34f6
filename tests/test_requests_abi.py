"""The calls that serve many requests in one step (norms of heads, adapters,
selection rules, token counts) refuse bad arguments on the host with the
documented codes (no CUDA call is made on these paths)."""
import ctypes

import pytest

from test_abi import FAKE, _status_codes, lib  # noqa: F401  (lib: the library fixture)
from test_attention_abi import batch, cache, ref, rotation

P, I, L, F, Z, U = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint)


class Norm(ctypes.Structure):
    _fields_ = [("weight", P), ("eps", F)]


class Adapters(ctypes.Structure):
    _fields_ = [("a", P), ("b", P), ("scale", P), ("a_adapter", L), ("b_adapter", L), ("adapters", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("slices", ctypes.c_int32),
                ("columns", ctypes.c_int32 * 4)]


class Rules(ctypes.Structure):
    _fields_ = [("counts", P), ("counts_stride", L), ("slot", P), ("repetition", P), ("presence", P), ("frequency", P),
                ("bias_offsets", P), ("bias_tokens", P), ("bias_values", P), ("allowed", P), ("allowed_stride", L),
                ("slots", ctypes.c_int32), ("bias_entries", ctypes.c_int32)]


def changed(s, kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def adapters(**kw):
    return changed(Adapters(FAKE, FAKE, FAKE, 4096, 4096, 3, 16, 64, 64, 2, (ctypes.c_int32 * 4)(40, 64, 0, 0)), kw)


def rules(**kw):
    return changed(Rules(FAKE, 1000, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 32, 4, 9), kw)


@pytest.fixture(scope="module")
def calls(lib):  # noqa: F811
    lib.f16_rope_ex.argtypes = [P, L, L, P, L, L, P, P, P, I, I, I, P]
    lib.f16_kv_append_ex.argtypes = [P, L, L, P, L, L, P, P, P, P, P, P, P, L, L, P, L, L, I, P]
    lib.f16_lora.argtypes = [P, L, P, L, P, L, P, P, I, P, Z, P]
    lib.f16_lora_workspace_bytes.argtypes = [P, I]
    lib.f16_lora_workspace_bytes.restype = Z
    lib.lm_head_argmax_topk_rules.argtypes = [P, P, P, P, I, I, I, I, I, P, P, P, P, Z, U, P]
    lib.w4_token_counts.argtypes = [P, L, I, I, P, P, P, I, I, U, P]
    return lib


C = _status_codes()


def workspace_bytes(calls, s, m):
    return calls.f16_lora_workspace_bytes(ref(s), m)   # (s lives through the call)


def test_rope_norm(calls):
    def rope(norm, r=None, x=FAKE, tokens=3, dim=64, xs=256):
        return calls.f16_rope_ex(x, xs, dim, FAKE, 256, dim, None, ref(r), ref(norm), tokens, 4, dim, None)
    assert rope(None) == C["W4_ERR_NULL"]
    assert rope(Norm(None, 1e-6)) == C["W4_ERR_NULL"]
    assert rope(Norm(FAKE + 4, 1e-6)) == C["W4_ERR_ALIGN"]
    for eps in (-1.0, float("nan"), float("inf")):
        assert rope(Norm(FAKE, eps)) == C["W4_ERR_SHAPE"], eps
    assert rope(Norm(FAKE, 0.0), tokens=-1) == C["W4_ERR_SHAPE"]
    assert rope(Norm(FAKE, 0.0), rotation(rot=72)) == C["W4_ERR_SHAPE"]
    assert rope(Norm(FAKE, 0.0), rotation(turns=None)) == C["W4_ERR_NULL"]
    assert rope(Norm(FAKE, 0.0), dim=264, xs=2112) == C["W4_ERR_SHAPE"]
    assert rope(Norm(FAKE, 0.0), x=None) == C["W4_ERR_NULL"]
    assert rope(Norm(FAKE, 0.0), xs=252) == C["W4_ERR_ALIGN"]
    assert rope(Norm(FAKE, 0.0), tokens=0, x=None) == C["W4A16_OK"]
    assert calls.f16_rope(FAKE, 256, 64, FAKE, 256, 64, None, None, 3, 4, 64, None) == C["W4_ERR_NULL"]


def test_append_norms(calls):
    def append(qn, kn, **kw):
        c, b = cache(), batch(**kw)
        return calls.f16_kv_append_ex(FAKE, 256, 128, FAKE, 256, 128, ref(c), ref(b), None, None, ref(qn), ref(kn),
                                      FAKE, 512, 128, FAKE, 512, 128, 4, None)
    for bad, code in ((Norm(None, 1e-6), "W4_ERR_NULL"), (Norm(FAKE, -1.0), "W4_ERR_SHAPE"), (Norm(FAKE + 8, 1e-6), "W4_ERR_ALIGN")):
        assert append(bad, None) == C[code]
        assert append(None, bad) == C[code]
        assert append(Norm(FAKE, 1e-6), bad) == C[code]
    assert append(Norm(FAKE, 1e-6), None, batch=0) == C["W4_ERR_SHAPE"]
    assert append(Norm(FAKE, 1e-6), None, total_q=0) == C["W4A16_OK"]


def test_lora(calls):
    big = 1 << 40

    def lora(s, m=5, x=FAKE, xs=64, y=FAKE, ys=64, out=FAKE, os=64, ids=FAKE, ws=FAKE, n=big):
        return calls.f16_lora(x, xs, y, ys, out, os, ref(s), ids, m, ws, n, None)
    assert lora(None) == C["W4_ERR_NULL"]
    for kw in (dict(adapters=0), dict(adapters=4097), dict(rank=0), dict(rank=12), dict(rank=136), dict(K=0), dict(K=60),
               dict(N=60), dict(N=0), dict(slices=0), dict(slices=5), dict(N=72), dict(slices=1),
               dict(columns=(ctypes.c_int32 * 4)(64, 64, 0, 0)), dict(columns=(ctypes.c_int32 * 4)(36, 64, 0, 0)),
               dict(columns=(ctypes.c_int32 * 4)(-8, 64, 0, 0))):
        assert lora(adapters(**kw)) == C["W4_ERR_SHAPE"], kw
        assert workspace_bytes(calls, adapters(**kw), 5) == 0, kw
    assert lora(adapters(), m=-1) == C["W4_ERR_SHAPE"]
    assert lora(adapters(), m=0, x=None, y=None, out=None, ids=None, ws=None, n=0) == C["W4A16_OK"]
    for kw in (dict(x=None), dict(y=None), dict(out=None), dict(ids=None)):
        assert lora(adapters(), **kw) == C["W4_ERR_NULL"], kw
    assert lora(adapters(a=None)) == lora(adapters(b=None)) == C["W4_ERR_NULL"]
    for kw in (dict(x=FAKE + 8), dict(y=FAKE + 2), dict(out=FAKE + 4), dict(ids=FAKE + 2), dict(xs=60), dict(ys=0), dict(os=-8),
               dict(ws=FAKE + 8)):
        assert lora(adapters(), **kw) == C["W4_ERR_ALIGN"], kw
    for kw in (dict(a=FAKE + 8), dict(b=FAKE + 8), dict(scale=FAKE + 2), dict(a_adapter=4), dict(b_adapter=0)):
        assert lora(adapters(**kw)) == C["W4_ERR_ALIGN"], kw
    need = workspace_bytes(calls, adapters(), 5)
    assert need >= 5 * 2 * 16 * 4
    assert lora(adapters(), ws=None) == lora(adapters(), n=need - 1) == C["W4_ERR_WORKSPACE"]


@pytest.mark.parametrize("m", [1, 32, 33, 1024, 1025, 70000])
def test_lora_workspace_holds_what_is_written(calls, m):
    """At least a share of h; with more than 64 ranks in all and more than 32 rows its fragments and their factors too."""
    for rank, slices, k in ((8, 1, 8), (16, 2, 2048), (24, 3, 2048), (128, 4, 11008)):
        ends = (ctypes.c_int32 * 4)(*(64 * (i + 1) for i in range(slices)))
        s = adapters(rank=rank, slices=slices, K=k, N=64 * slices, columns=ends)
        need = workspace_bytes(calls, s, m)
        least = m * rank * slices * 4
        if m > 32 and rank * slices > 64:
            padded = 32 if rank <= 32 else 128
            least += m * padded * slices * 4 + m * 4
        assert least <= need <= 8 * least + 64
    assert workspace_bytes(calls, adapters(), 0) == workspace_bytes(calls, None, 5) == 0


def test_lora_rows_of_out_do_not_overlap(calls):
    s = adapters()
    for os, m, code in ((56, 2, "W4_ERR_SHAPE"), (8, 5, "W4_ERR_SHAPE"), (56, 1, "W4_ERR_WORKSPACE"), (64, 2, "W4_ERR_WORKSPACE")):
        assert calls.f16_lora(FAKE, 64, FAKE, 64, FAKE, os, ref(s), FAKE, m, None, 0, None) == C[code], (os, m)


def test_lora_workspace_grows_with_the_rows(calls):
    for rank, slices, k in ((8, 1, 64), (16, 3, 2048), (32, 2, 896), (64, 3, 2048), (128, 4, 11008)):
        ends = (ctypes.c_int32 * 4)(*(64 * (i + 1) for i in range(slices)))
        s = adapters(rank=rank, slices=slices, K=k, N=64 * slices, columns=ends)
        sizes = [workspace_bytes(calls, s, m) for m in (*range(1, 2200), 4096, 4097, 65536, 70001, 1 << 20)]
        assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_rules(calls):
    def pick(r, ws=FAKE, n=1 << 30, flags=0, N=1000, idx=FAKE):
        return calls.lm_head_argmax_topk_rules(FAKE, FAKE, FAKE, FAKE, 2, N, 64, 64, 5, idx, FAKE, ref(r), ws, n, flags, None)
    for kw, code in ((dict(slot=None), "W4_ERR_NULL"), (dict(slots=0), "W4_ERR_SHAPE"), (dict(counts_stride=999), "W4_ERR_SHAPE"),
                     (dict(counts=FAKE + 1), "W4_ERR_ALIGN"), (dict(slot=FAKE + 2), "W4_ERR_ALIGN"),
                     (dict(repetition=FAKE + 2), "W4_ERR_ALIGN"), (dict(presence=FAKE + 1), "W4_ERR_ALIGN"),
                     (dict(frequency=FAKE + 3), "W4_ERR_ALIGN"), (dict(bias_tokens=None), "W4_ERR_NULL"),
                     (dict(bias_values=None), "W4_ERR_NULL"), (dict(bias_entries=-1), "W4_ERR_SHAPE"),
                     (dict(bias_entries=(1 << 30) + 1), "W4_ERR_SHAPE"), (dict(bias_offsets=FAKE + 2), "W4_ERR_ALIGN"),
                     (dict(bias_values=FAKE + 2), "W4_ERR_ALIGN"), (dict(allowed_stride=31), "W4_ERR_SHAPE"),
                     (dict(allowed=FAKE + 2), "W4_ERR_ALIGN")):
        assert pick(rules(**kw)) == C[code], kw
    assert pick(rules(), flags=2) == C["W4_ERR_SHAPE"]
    assert pick(rules(), ws=None) == pick(rules(), n=16) == C["W4_ERR_WORKSPACE"]
    assert pick(rules(), ws=FAKE + 8) == C["W4_ERR_ALIGN"]
    assert pick(rules(), idx=None) == C["W4_ERR_NULL"]
    assert pick(None, N=4) == C["W4_ERR_SHAPE"]
    # parts that are left out are not looked at
    assert pick(rules(counts=None, slots=0, slot=None), ws=None) == C["W4_ERR_WORKSPACE"]
    assert pick(rules(bias_offsets=None, bias_entries=-5), ws=None) == C["W4_ERR_WORKSPACE"]
    assert pick(rules(allowed=None, allowed_stride=0), ws=None) == C["W4_ERR_WORKSPACE"]


def test_token_counts(calls):
    def count(counts=FAKE, stride=1000, slots=4, n=1000, slot=FAKE, tokens=FAKE, offsets=FAKE, batch=2, total=5, flags=0):
        return calls.w4_token_counts(counts, stride, slots, n, slot, tokens, offsets, batch, total, flags, None)
    for kw, code in ((dict(counts=None), "W4_ERR_NULL"), (dict(slot=None), "W4_ERR_NULL"), (dict(tokens=None), "W4_ERR_NULL"),
                     (dict(slots=0), "W4_ERR_SHAPE"), (dict(n=0), "W4_ERR_SHAPE"), (dict(stride=999), "W4_ERR_SHAPE"),
                     (dict(batch=-1), "W4_ERR_SHAPE"), (dict(batch=65536), "W4_ERR_SHAPE"), (dict(total=-1), "W4_ERR_SHAPE"),
                     (dict(offsets=None), "W4_ERR_SHAPE"), (dict(flags=4), "W4_ERR_SHAPE"), (dict(counts=FAKE + 1), "W4_ERR_ALIGN"),
                     (dict(slot=FAKE + 2), "W4_ERR_ALIGN"), (dict(tokens=FAKE + 1), "W4_ERR_ALIGN"),
                     (dict(offsets=FAKE + 2), "W4_ERR_ALIGN")):
        assert count(**kw) == C[code], kw
    assert count(total=0, tokens=None) == C["W4A16_OK"]
    assert count(batch=0, total=0, tokens=None, flags=2) == C["W4A16_OK"]


def test_no_sequences_to_count(calls):
    """Empty arrays have no address."""
    for flags in (0, 1, 2, 3):
        for offsets in (FAKE, None):
            assert calls.w4_token_counts(FAKE, 1000, 4, 1000, None, None, offsets, 0, 0, flags, None) == C["W4A16_OK"]
