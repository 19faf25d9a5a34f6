"""A decoder layer's attention block on int4 weights: q/k/v projections, rotary
positions, a paged cache, attention over it, o projection; norms of the query
and key heads and low-rank adapters of each request where the block has them.

Four prompts of different lengths go in as one batch (their projections
dequantised once, or through the int4 GEMM up to 128 tokens), then single
tokens are decoded by one captured graph whose batch lives on the device.
Synthetic weights of the Qwen2.5-3B shapes (hidden 2048, 16 query and 2
key/value heads of 128).

    python examples/attention_block.py
"""
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import int4_weight_only_affine_gb300 as w4  # noqa: E402
import synth  # noqa: E402


class AttentionBlock:
    """The block and its cache.  The projections of q, k and v are one weight.
    norms: normalise the query and key heads; adapters: how many requests can
    choose from, of this rank."""

    def __init__(self, hidden=2048, q_heads=16, kv_heads=2, dim=128, pages=256, page_size=16, max_tokens=512,
                 base=1e6, seed=0, device="cuda", norms=False, adapters=0, rank=16):
        self.hidden, self.q_heads, self.kv_heads, self.dim, self.page_size = hidden, q_heads, kv_heads, dim, page_size
        self.qkv = self._weight(seed, (q_heads + 2 * kv_heads) * dim, hidden, device)
        self.o = self._weight(seed + 1, hidden, q_heads * dim, device)
        shape = (pages, page_size, kv_heads, dim)
        self.cache = w4.KVCache(*(torch.zeros(shape, dtype=torch.float16, device=device) for _ in range(2)))
        self.rope = w4.Rope(*w4.rope_turns(dim, base=base, device=device))
        self.workspace = w4.attention_workspace(self.cache, q_heads, max_tokens)
        gen = torch.Generator(device=device).manual_seed(seed)
        self.q_norm = self.k_norm = self.qkv_adapters = self.o_adapters = None
        if norms:
            self.q_norm, self.k_norm = (w4.HeadNorm(1 + 0.2 * torch.randn(dim, generator=gen, device=device)) for _ in range(2))
        if adapters:
            self.qkv_adapters = self._adapters(gen, adapters, rank, hidden, [q_heads * dim, kv_heads * dim, kv_heads * dim])
            self.o_adapters = self._adapters(gen, adapters, rank, q_heads * dim, [hidden])

    @staticmethod
    def _adapters(gen, n, rank, k, columns):
        a, b = (torch.randn(*shape, generator=gen, device=gen.device) for shape in
                ((n, len(columns), rank, k), (n, sum(columns), rank)))
        return w4.Adapters((a * k**-0.5).half(), (b * 0.1).half(), columns=columns)

    @staticmethod
    def _weight(seed, n, k, device):
        qw, s, b = synth.make_linear(seed, n, k)
        # Scales of trained layers: outputs of the order of the inputs.
        s, b = (s / np.float16(8)).astype(np.float16), (b / np.float16(8)).astype(np.float16)
        return [torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).to(device) for a in (qw, s, b)]

    @staticmethod
    def _project(x, weight):
        if x.shape[0] <= 16:
            return w4.w4_gemv(x, *weight)
        if x.shape[0] <= 128:
            return w4.w4_gemm(x, *weight)
        return w4.f16_gemm(x, w4.w4_dequant_f16(*weight))

    def __call__(self, x, batch, ids=None):
        """x [tokens][hidden]: the new tokens of the batch's sequences, one after the other;
        ids int32 [tokens]: the adapter of each (negative: none)."""
        n, hq, hk, d = x.shape[0], self.q_heads, self.kv_heads, self.dim
        qkv = self._project(x, self.qkv)
        if ids is not None:
            w4.f16_lora(x, self.qkv_adapters, ids, qkv)
        qkv = qkv.view(n, hq + 2 * hk, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        w4.f16_kv_append(k, v, self.cache, batch, rope=self.rope, q=q, y=q, q_norm=self.q_norm, k_norm=self.k_norm)
        y = w4.f16_attention(q, self.cache, batch, workspace=self.workspace).view(n, hq * d)
        out = self._project(y, self.o)
        return out if ids is None else w4.f16_lora(y, self.o_adapters, ids, out)


def page_table(lengths, page_size, pages, seed=0):
    """int32 [sequences][pages]: pages for `lengths` positions of each, in no order."""
    need = [-(-n // page_size) for n in lengths]
    order = np.random.RandomState(seed).permutation(pages)
    table = np.full((len(lengths), max(need)), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table


def main(prompts=(300, 17, 120, 63), steps=64):
    block = AttentionBlock()
    table = torch.from_numpy(page_table([n + steps for n in prompts], block.page_size, block.cache.num_pages)).cuda()
    n = len(prompts)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")

    offsets = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]), dtype=torch.int32, device="cuda")
    x = torch.randn(sum(prompts), block.hidden, device="cuda").half()
    y = block(x, w4.KVBatch(table, offsets, lens, sum(prompts), max(prompts)))
    print(f"prompts of {prompts} tokens: output {tuple(y.shape)}")

    # Decode: one new token of each sequence a step; the graph moves the lengths on itself.
    one = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    batch = w4.KVBatch(table, one, lens, n, 1)
    x = torch.randn(n, block.hidden, device="cuda").half()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # once outside the capture: kernels are set up on their first launch
        lens.add_(1)
        block(x, batch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens.add_(1)
        y = block(x, batch)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / (steps - 1)
    assert w4.device_status() == 0
    print(f"decode of {n} sequences up to {lens.tolist()} tokens: {t * 1e6:.1f} us a step of this block")
    return y


if __name__ == "__main__":
    main()
