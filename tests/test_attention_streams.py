"""What the attention calls make for a call on another stream than the current one belongs to that stream (CPU: the
library and the streams are stand-ins)."""
import contextlib
import os
import types

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")


@pytest.fixture()
def att(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "int4_weight_only_affine_gb300", "libw4a16.so")):
        import __graft_entry__
        __graft_entry__.build()
    from int4_weight_only_affine_gb300 import attention as att
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
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: state.stream)
    monkeypatch.setattr(torch, "empty", maker(torch.empty))
    monkeypatch.setattr(torch, "zeros", maker(torch.zeros))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state.kept.append(s))
    monkeypatch.setattr(att, "lib", types.SimpleNamespace(f16_rope=called, f16_kv_append=called, f16_attention=called,
                                                          f16_attention_workspace_bytes=lambda *a: 64))
    monkeypatch.setattr(att, "_heads", lambda t, name: (16, 8, 8))
    monkeypatch.setattr(att, "_dev", lambda t, name, dtypes: 16)
    monkeypatch.setattr(att, "_stream", lambda s: 0)
    att_cache = types.SimpleNamespace(heads=2, head_dim=64, ptr=0, k=torch.ones(1))
    att_batch = types.SimpleNamespace(total_q=3, max_q_len=3, ptr=0)
    return att, att_cache, att_batch, state


@pytest.mark.parametrize("stream", [None, "side"])
def test_memory_belongs_to_the_stream_of_the_call(att, stream):
    att, cache, batch, state = att
    q, k = torch.ones(3, 4, 64).half(), torch.ones(3, 2, 64).half()
    rope = types.SimpleNamespace(ptr=0)
    owner = stream or "current"
    att.f16_attention(q, cache, batch, stream=stream)
    assert state.made == [owner, owner]   # y and the zero-filled workspace
    state.made.clear()
    att.f16_attention(q, cache, batch, y=q, stream=stream)
    assert state.made == [owner]
    state.made.clear()
    att.f16_rope(q, rope, stream=stream)
    att.f16_kv_append(k, k, cache, batch, rope=rope, q=q, stream=stream)
    assert state.made == [owner, owner]
    # outputs are kept for the current stream's work on them
    assert state.kept == ([] if stream is None else ["current"] * 3)
