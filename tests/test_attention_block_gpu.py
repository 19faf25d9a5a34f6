"""The projections, rotation, cache and attention together, as examples/attention_block.py runs them."""
import importlib.util
import os

import numpy as np
import pytest

from _attn import rotate, thetas
from _gpu import require_gpu
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense(block, xs):
    """The block's outputs for the whole of each sequence, by its definition in binary64."""
    def weight(w):
        qw, s, b = (t.cpu().numpy() for t in w)
        codes = (qw.view(np.uint32)[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
        return codes.reshape(qw.shape[0], -1) * np.repeat(s.astype(np.float64), 64, 1) + np.repeat(b.astype(np.float64), 64, 1)
    wq, wo = weight(block.qkv), weight(block.o)
    hq, hk, d = block.q_heads, block.kv_heads, block.dim
    out = []
    for x in xs:
        n = len(x)
        qkv = (x.astype(np.float64) @ wq.T).reshape(n, hq + 2 * hk, d)
        r = rotate(qkv[:, :hq + hk], np.arange(n), thetas(d, 1e6))
        y = np.zeros((n, hq, d))
        for h in range(hq):
            s = r[:, h] @ r[:, hq + h * hk // hq].T / np.sqrt(d)
            s[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            y[:, h] = p @ qkv[:, hq + hk + h * hk // hq] / p.sum(1, keepdims=True)
        out.append(y.reshape(n, hq * d) @ wo.T)
    return out


def test_prompt_chunks_and_single_tokens_give_the_dense_block(example):
    """Prompts in one batch, a second chunk of one of them with single tokens of the others, then single tokens."""
    import torch

    import int4_weight_only_affine_gb300 as w4
    block = example.AttentionBlock(hidden=512, q_heads=4, kv_heads=2, dim=64, pages=64, max_tokens=200)
    final = [160, 40, 9]
    g = np.random.RandomState(0)
    xs = [g.standard_normal((n, 512)).astype(np.float16) for n in final]
    want = dense(block, xs)
    table = torch.from_numpy(example.page_table(final, 16, 64)).cuda()
    done, got = [0, 0, 0], [[], [], []]
    for news in ([60, 33, 2], [97, 1, 1], [1, 1, 1], [1, 1, 1], [1, 4, 4]):
        x = np.concatenate([xs[b][done[b]:done[b] + k] for b, k in enumerate(news)])
        done = [a + k for a, k in zip(done, news)]
        offs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        batch = w4.KVBatch(table, torch.from_numpy(offs).cuda(), torch.tensor(done, dtype=torch.int32, device="cuda"),
                           len(x), max(news))
        y = block(torch.from_numpy(x).cuda(), batch).cpu().numpy()
        for b in range(3):
            got[b].append(y[offs[b]:offs[b + 1]])
    assert done == final and w4.device_status() == 0
    for b in range(3):
        y, w = np.concatenate(got[b]).astype(np.float64), want[b]
        # Five roundings to binary16 on the way (qkv, rotated q and k, probabilities, attention, output), each
        # 2**-11 of its operand; they reach the output, a sum of 256 products, as independent errors: a few
        # thousandths of its size in norm, and of its rms elementwise.
        assert np.linalg.norm(y - w) <= 4e-3 * np.linalg.norm(w)
        assert np.abs(y - w).max() <= 2e-2 * np.sqrt(np.mean(w * w)) + 2.0**-10 * np.abs(w).max()


def test_example_runs(example):
    y = example.main(prompts=(40, 3), steps=5)
    assert bool(y.isfinite().all())
