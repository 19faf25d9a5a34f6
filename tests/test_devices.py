"""Calls whose tensors are not on the current device are refused before anything is launched (CPU: the tensors only say
that they are on a GPU)."""
import os
import types

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")


class Elsewhere(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))

    def get_device(self):
        return 1


def elsewhere(*shape, dtype=torch.float16):
    return torch.ones(*shape, dtype=dtype).as_subclass(Elsewhere)


@pytest.fixture()
def w4(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "int4_weight_only_affine_gb300", "libw4a16.so")):
        import __graft_entry__
        __graft_entry__.build()
    import int4_weight_only_affine_gb300 as w4
    monkeypatch.setattr(w4, "_current_device", lambda: 0)
    return w4


def test_tensors_of_another_device_are_refused(w4):
    x, heads = elsewhere(3, 64), elsewhere(3, 2, 64)
    qw, s = elsewhere(8, 8, dtype=torch.int32), elsewhere(8, 1)
    ints = elsewhere(3, dtype=torch.int32)
    rope = types.SimpleNamespace(ptr=0)
    cache = types.SimpleNamespace(heads=2, head_dim=64, ptr=0, k=heads)
    batch = types.SimpleNamespace(total_q=3, max_q_len=3, ptr=0)
    adapters = types.SimpleNamespace(K=64, N=64, ptr=0, sized=None, device=x.device)
    counts = types.SimpleNamespace(counts=elsewhere(2, 9, dtype=torch.int16), ptr=0, stride=9, slots=2, vocabulary=9)
    for call in (lambda: w4.w4_gemv(x, qw, s, s), lambda: w4.lm_head_argmax_topk(x, qw, s, s),
                 lambda: w4.w4_dequant_f16(qw, s, s), lambda: w4.w4_gemm(x, qw, s, s), lambda: w4.f16_gemm(x, elsewhere(64, 8)),
                 lambda: w4.GemvList([(x, qw, s, s, x, False)]).run(elsewhere(64, dtype=torch.uint8)),
                 lambda: w4.f16_rope(heads, rope), lambda: w4.f16_kv_append(heads, heads, cache, batch),
                 lambda: w4.f16_attention(heads, cache, batch), lambda: w4.f16_lora(x, adapters, ints, x),
                 lambda: w4.token_counts_add(counts, ints, ints)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_adapters_of_another_device_are_refused(w4, monkeypatch):
    monkeypatch.setattr(w4, "_current_device", lambda: 1)
    adapters = types.SimpleNamespace(K=64, N=64, ptr=0, sized=None, device=torch.device("cuda", 0))
    x = elsewhere(3, 64)
    with pytest.raises(ValueError, match="adapters on cuda:0"):
        w4.f16_lora(x, adapters, elsewhere(3, dtype=torch.int32), x)
