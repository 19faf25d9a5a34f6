"""Norms, adapters, selection rules and token counts in one decoding loop of different requests, as a server runs them
(the block of examples/attention_block.py, then the LM head), against binary64."""
import numpy as np
import pytest

import synth
from _attn import rotate, thetas
from _gpu import require_gpu, to_dev
from test_attention_block_gpu import example  # noqa: F401  (the example module)

pytestmark = pytest.mark.gpu
EPS = 1e-6


def dense(block, xs, ids):
    """The block's outputs for the whole of each sequence under its adapter, by its definition in binary64."""
    def weight(w, adapters, i):
        qw, s, b = (t.cpu().numpy() for t in w)
        codes = (qw.view(np.uint32)[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
        full = codes.reshape(qw.shape[0], -1) * np.repeat(s.astype(np.float64), 64, 1) + np.repeat(b.astype(np.float64), 64, 1)
        if i >= 0:
            at = 0
            a, b = (t.cpu().numpy().astype(np.float64) for t in (adapters.a, adapters.b))
            for j in range(adapters.struct.slices):
                end = adapters.struct.columns[j]
                full[at:end] += b[i, at:end] @ a[i, j]
                at = end
        return full

    hq, hk, d = block.q_heads, block.kv_heads, block.dim
    nq, nk = (m.weight.cpu().numpy().astype(np.float64) for m in (block.q_norm, block.k_norm))
    out = []
    for x, i in zip(xs, ids):
        n = len(x)
        qkv = (x.astype(np.float64) @ weight(block.qkv, block.qkv_adapters, i).T).reshape(n, hq + 2 * hk, d)
        z = qkv[:, :hq + hk] / np.sqrt((qkv[:, :hq + hk] ** 2).mean(-1, keepdims=True) + EPS)
        z[:, :hq] *= nq
        z[:, hq:] *= nk
        r = rotate(z, np.arange(n), thetas(d, 1e6))
        y = np.zeros((n, hq, d))
        for h in range(hq):
            s = r[:, h] @ r[:, hq + h * hk // hq].T / np.sqrt(d)
            s[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            y[:, h] = p @ qkv[:, hq + hk + h * hk // hq] / p.sum(1, keepdims=True)
        out.append(y.reshape(n, hq * d) @ weight(block.o, block.o_adapters, i).T)
    return out


def test_block_with_norms_and_adapters(example):  # noqa: F811
    """Prompts in one batch, chunks beside single tokens, then single tokens, each sequence under its own adapter."""
    import torch

    import int4_weight_only_affine_gb300 as w4
    block = example.AttentionBlock(hidden=512, q_heads=4, kv_heads=2, dim=64, pages=64, max_tokens=200, norms=True, adapters=3)
    final, ids = [160, 40, 9], [2, -1, 0]
    g = np.random.RandomState(0)
    xs = [g.standard_normal((n, 512)).astype(np.float16) for n in final]
    want = dense(block, xs, ids)
    table = torch.from_numpy(example.page_table(final, 16, 64)).cuda()
    done, got = [0, 0, 0], [[], [], []]
    for news in ([60, 33, 2], [97, 1, 1], [1, 1, 1], [1, 1, 1], [1, 4, 4]):
        x = np.concatenate([xs[b][done[b]:done[b] + k] for b, k in enumerate(news)])
        done = [a + k for a, k in zip(done, news)]
        offs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        batch = w4.KVBatch(table, to_dev(offs), to_dev(np.array(done, np.int32)), len(x), max(news))
        y = block(to_dev(x), batch, to_dev(np.repeat(np.array(ids, np.int32), news))).cpu().numpy()
        for b in range(3):
            got[b].append(y[offs[b]:offs[b + 1]])
    assert done == final and w4.device_status() == 0
    for b in range(3):
        y, w = np.concatenate(got[b]).astype(np.float64), want[b]
        # Seven roundings to binary16 on the way (qkv, its sum with the adapter, normed and rotated q and k,
        # probabilities, attention, output and its sum), each 2**-11 of its operand; they reach the output, a sum
        # of 256 products, as independent errors: a few thousandths of its size in norm, and of its rms elementwise.
        assert np.linalg.norm(y - w) <= 5e-3 * np.linalg.norm(w)
        assert np.abs(y - w).max() <= 2.5e-2 * np.sqrt(np.mean(w * w)) + 2.0**-10 * np.abs(w).max()


def test_decoding_loop_in_a_graph(example):  # noqa: F811
    """Greedy steps of four requests (one slot empty) captured once: adapters, penalties and masks differ by request, the
    selected tokens are counted and embedded on the device.  Each step's selection is checked from the hidden states
    that the GPU had; the counts are checked exactly; a replay from the start gives the same tokens."""
    import torch

    import int4_weight_only_affine_gb300 as w4
    hidden, vocab, n, steps = 512, 1000, 4, 7
    block = example.AttentionBlock(hidden=hidden, q_heads=4, kv_heads=2, dim=64, pages=64, norms=True, adapters=3)
    qw, s, b = synth.make_linear(7, vocab, hidden)
    head = [to_dev(a) for a in (qw, s, b)]
    codes = (qw[:, :, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
    wfull = codes.reshape(vocab, -1) * np.repeat(s.astype(np.float64), 64, 1) + np.repeat(b.astype(np.float64), 64, 1)
    g = np.random.RandomState(3)
    embed = to_dev(g.standard_normal((vocab + 1, hidden)).astype(np.float16))
    allowed = g.random_sample((n, vocab)) < 0.5
    allowed[1] = True
    words = np.zeros((n, 1024), bool)
    words[:, :vocab] = allowed
    bits = np.packbits(words.reshape(n, 32, 32), axis=2, bitorder="little").view(np.uint32).reshape(n, 32)
    slots = np.array([5, 0, 3, -1], np.int32)
    rep, pres, freq = (np.array(v, np.float32) for v in ([1.5, 1.0, 1.2, 2.0], [0.5, 0.0, 1.0, 9.0], [0.25, 0.5, 0.0, 9.0]))
    counts = w4.TokenCounts.new(6, vocab)
    rules = w4.LogitRules(counts, to_dev(slots), to_dev(rep), to_dev(pres), to_dev(freq), allowed=to_dev(bits))
    prompt = g.randint(0, vocab, 60).astype(np.int32)
    offsets = np.array([0, 25, 40, 60, 60], np.int32)
    ids = to_dev(np.array([1, -1, 2, 0], np.int32))
    table = torch.from_numpy(example.page_table([steps + 2] * n, 16, 64)).cuda()
    lens, one = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n + 1, dtype=torch.int32, device="cuda")
    batch = w4.KVBatch(table, one, lens, n, 1)
    x = torch.zeros(n, hidden, dtype=torch.float16, device="cuda")
    y, idx, val = (torch.zeros(n, hidden, dtype=torch.float16, device="cuda"),
                   torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, 1, device="cuda"))
    ws = torch.empty(w4.lm_head_workspace_bytes(n, vocab, 1), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        y.copy_(block(x, batch, ids))
        w4.lm_head_argmax_topk(y, *head, k=1, idx=idx, val=val, workspace=ws, rules=rules)
        w4.token_counts_add(counts, rules.tensors[1], idx.view(-1))
        x.copy_(embed[idx.view(-1).long()])

    def start():
        lens.zero_()
        x.copy_(embed[:n])
        w4.token_counts_add(counts, rules.tensors[1], to_dev(prompt), to_dev(offsets), prompt=True, reset=True)

    start()
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    runs = []
    for _ in range(2):
        start()
        seen = np.zeros((6, vocab), np.uint16)
        for i in range(3):
            seen[slots[i], prompt[offsets[i]:offsets[i + 1]]] |= 0x8000
        tokens = []
        for _ in range(steps):
            graph.replay()
            torch.cuda.synchronize()
            hidden_states, pick = y.cpu().numpy().astype(np.float64), idx.cpu().numpy()[:, 0]
            logits, room = hidden_states @ wfull.T, np.abs(hidden_states) @ np.abs(wfull).T
            for r in range(n):
                z = logits[r].copy()
                if slots[r] >= 0:
                    c = seen[slots[r]]
                    z = np.where(c > 0, np.where(z > 0, z / rep[r], z * rep[r]), z)
                    t = (c & 0x7FFF).astype(np.float64)
                    z = z - freq[r] * t - pres[r] * (t > 0)
                z[~allowed[r]] = -np.inf
                # the GEMV's bound on logits, times the most that a penalty scales by
                tol = 2.0 * (1e-3 * room[r].max() + 1e-3) * 1.5
                assert allowed[r, pick[r]] and z[pick[r]] >= z.max() - tol
                assert abs(float(val[r, 0]) - z[pick[r]]) <= tol
                if slots[r] >= 0:
                    seen[slots[r], pick[r]] += 1
            assert np.array_equal(counts.counts.cpu().numpy().view(np.uint16)[[0, 3, 5]], seen[[0, 3, 5]])
            tokens.append(pick.tolist())
        runs.append(tokens)
    assert runs[0] == runs[1] and w4.device_status() == 0
    assert len({tuple(t) for t in zip(*runs[0])}) > 1   # requests differ
