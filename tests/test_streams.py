"""What the projection and selection calls make for a call on another stream than the current one belongs to that
stream (CPU: the library and the streams are stand-ins)."""
import contextlib
import os
import types

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")


@pytest.fixture()
def w4(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "int4_weight_only_affine_gb300", "libw4a16.so")):
        import __graft_entry__
        __graft_entry__.build()
    import int4_weight_only_affine_gb300 as w4
    state = types.SimpleNamespace(stream="current", made=[], kept=[])

    @contextlib.contextmanager
    def on(stream):
        state.stream, before = stream, state.stream
        yield
        state.stream = before

    def maker(fn):
        def make(*shape, dtype, device):
            state.made.append(state.stream)
            return fn(*shape, dtype=dtype)
        return make

    called = lambda *a: 0  # noqa: E731
    size = lambda *a: 64  # noqa: E731
    copy = torch.Tensor.reshape

    def reshape(t, *shape):
        if not t.is_contiguous():
            state.made.append(state.stream)
        return copy(t, *shape)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: state.stream)
    monkeypatch.setattr(torch, "empty", maker(torch.empty))
    monkeypatch.setattr(torch, "zeros", maker(torch.zeros))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state.kept.append(s))
    monkeypatch.setattr(torch.Tensor, "reshape", reshape)
    monkeypatch.setattr(w4, "lib", types.SimpleNamespace(
        w4_gemv_ex=called, w4_gemv_seq=called, lm_head_argmax_topk_ex=called, lm_head_argmax_topk_rules=called,
        w4_dequant_f16_ex=called, w4_gemm_ex=called, f16_gemm_ex=called, lm_head_workspace_bytes=size,
        w4_gemm_workspace_bytes=size, w4_gemv_seq_workspace_bytes_ex=size))
    monkeypatch.setattr(w4, "_dev", lambda t, name, dtypes: 16)
    monkeypatch.setattr(w4, "_stream", lambda s: 0)
    return w4, state


@pytest.mark.parametrize("stream", [None, "side"])
def test_memory_belongs_to_the_stream_of_the_call(w4, stream):
    w4, state = w4
    owner = stream or "current"
    x, qw = torch.ones(3, 64).half(), torch.ones(8, 8, dtype=torch.int32)
    s = torch.ones(8, 1).half()
    apart = torch.ones(3, 64, 1).half().expand(3, 64, 2).transpose(1, 2)     # [3][2][64], rows that a copy brings together
    rules = types.SimpleNamespace(_of=lambda rows, tokens: 16)

    def made(call, what):
        state.made.clear()
        state.kept.clear()
        call()
        assert state.made == [owner] * what
        return list(state.kept)

    def outputs(call, count, more=0):
        assert made(call, count + more) == ([] if stream is None else ["current"] * count)
    outputs(lambda: w4.w4_gemv(x, qw, s, s, stream=stream), 1)
    outputs(lambda: w4.w4_gemv(apart, qw, s, s, stream=stream), 1, 1)
    outputs(lambda: w4.lm_head_argmax_topk(x, qw, s, s, k=2, stream=stream), 2, 1)
    outputs(lambda: w4.lm_head_argmax_topk(x, qw, s, s, k=2, stream=stream, rules=rules), 2, 1)
    outputs(lambda: w4.w4_dequant_f16(qw, s, s, stream=stream), 1)
    outputs(lambda: w4.w4_gemm(x, qw, s, s, stream=stream), 1, 1)
    outputs(lambda: w4.f16_gemm(x, torch.ones(64, 8).half(), stream=stream), 1)
    outputs(lambda: w4.w4_gemv_seq([(x, qw, s, s, x, False)], stream=stream), 0, 1)


def test_a_list_takes_no_copy_of_its_activations(w4):
    """A list keeps addresses: an x that only a copy could bring into rows is refused."""
    w4, state = w4
    qw, s = torch.ones(8, 8, dtype=torch.int32), torch.ones(8, 1).half()
    apart = torch.ones(3, 64, 1).half().expand(3, 64, 2).transpose(1, 2)
    with pytest.raises(ValueError):
        w4.GemvList([(apart, qw, s, s, torch.ones(6, 8).half(), False)])
    assert w4.GemvList([(torch.ones(3, 2, 64).half(), qw, s, s, torch.ones(6, 8).half(), False)]).M == 6


def test_activations_and_outputs_too_small_are_refused(w4):
    w4, state = w4
    x, qw, s = torch.ones(3, 64).half(), torch.ones(8, 8, dtype=torch.int32), torch.ones(8, 1).half()
    few, ints, floats = torch.ones(23).half(), torch.ones(5, dtype=torch.int32), torch.ones(5)
    w16 = torch.ones(64, 8).half()
    narrow, y = torch.ones(3, 56).half(), torch.ones(3, 8).half()
    gemv = lambda x=x, y=y: w4.w4_gemv(x, qw, s, s, y=y)  # noqa: E731
    gemm = lambda x=x, y=y: w4.w4_gemm(x, qw, s, s, y=y)  # noqa: E731
    dense = lambda x=x, y=y: w4.f16_gemm(x, w16, y=y)  # noqa: E731
    listed = lambda x=x, y=y: w4.GemvList([(x, qw, s, s, y, False)])  # noqa: E731
    pick = lambda x=x, **kw: w4.lm_head_argmax_topk(x, qw, s, s, k=2, **kw)  # noqa: E731
    for call in (gemv, gemm, dense, listed, pick):
        call()
        with pytest.raises(ValueError):
            call(x=narrow)
    for call in (gemv, gemm, dense, listed):
        with pytest.raises(ValueError):
            call(y=few)
    for kw in (dict(idx=ints), dict(val=floats)):
        with pytest.raises(ValueError):
            pick(**kw)
    with pytest.raises(ValueError):
        w4.w4_dequant_f16(qw, s, s, w16=torch.ones(511).half())
    assert w4.w4_gemv(x, qw, s, s, y=torch.ones(40).half()).shape == (40,)    # room enough
