"""Cases of the operators that serve many different requests in one step, with their plain forms.

Norm of every query and key head with the rotation in the same pass (f16_rope
and f16_kv_append with norms), low-rank adapters of many requests beside a
shared projection (f16_lora), token selection under penalties, biases and masks
(lm_head_argmax_topk with rules) and the token counts that these read
(token_counts_add).  With own = False run() computes them with elementary torch
operations in 32 bits, with own = True by the framework's calls.  exact()
restates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
BASE = 1000000.0  # base of the rotation's wavelengths
EPS = 1e-6        # of the head norms
VOCAB = 151936
PROMPT = 1 << 15  # bit of a count that marks a token of the prompt


# ---------------------------------------------------------------- the cases

def _rope(name, tokens, heads, d, rot, interleaved):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": heads, "d": d, "rot": rot, "interleaved": interleaved}


def _append(name, batch, q, ctx, hq, hkv, d, page, rot, interleaved, ragged):
    return {"name": name, "op": "append", "batch": batch, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "rot": rot, "interleaved": interleaved, "ragged": ragged}


def _lora(name, rows, sequences, adapters, rank, k, columns, none, layout):
    """columns: widths of the column slices, joined by "+"; none: share of rows or sequences without an adapter."""
    return {"name": name, "op": "lora", "rows": rows, "sequences": sequences, "adapters": adapters, "rank": rank,
            "k": k, "columns": columns, "none": none, "layout": layout}


def _pick(name, rows, n, k, top, seen, masked, biases, symmetric):
    return {"name": name, "op": "pick", "rows": rows, "n": n, "k": k, "top": top, "seen": seen, "masked": masked,
            "biases": biases, "symmetric": symmetric}


def _seen(name, slots, batch, tokens, n, reset, ragged):
    return {"name": name, "op": "seen", "slots": slots, "batch": batch, "tokens": tokens, "n": n, "reset": reset,
            "ragged": ragged}


def listed():
    return [
        # Queries of a long prompt, normed and half of each head rotated: bandwidth.
        _rope("norm_rope_prompt", 16384, 16, 128, 64, True),
        # One decode step of 16 sequences, 16 query and 8 key/value heads of 128: latency.
        _append("norm_append_step", 16, 1, 2000, 16, 8, 128, 16, 128, False, 3),
        # Prompts of up to 4096 tokens, 14 query and 2 key/value heads of 64: bandwidth.
        _append("norm_append_prompts", 8, 4096, 6000, 14, 2, 64, 64, 64, False, 5),
        # q|k|v of eight decoding requests with four adapters, some without: latency.
        _lora("lora_step", 8, 8, 4, 16, 2048, "2048+256+256", 0.15, "rows"),
        # The down projection of a full decoding batch with many adapters: their bytes.
        _lora("lora_batch", 64, 64, 32, 32, 11008, "2048", 0.1, "rows"),
        # gate|up of one prompt of 1570 tokens under one adapter: bandwidth of the projection's output.
        _lora("lora_prompt", 1570, 1, 8, 16, 2048, "11008+11008", 0.0, "sequences"),
        # q|k|v of six prompts, with adapters of high rank, some without: bandwidth and arithmetic.
        _lora("lora_prompts", 4096, 6, 8, 64, 2048, "2048+256+256", 0.3, "sequences"),
        # A small classifying head, best five of 1000, four requests: latency.
        _pick("pick_small", 4, 1000, 896, 5, 0.2, True, 8, False),
        # Greedy decoding of one request with penalties over the full vocabulary.
        _pick("pick_step", 1, VOCAB, 1024, 1, 0.03, False, 0, False),
        # Sixteen requests, best 50 each, with penalties, biases and grammar masks, one of which allows nothing.
        _pick("pick_batch", 16, VOCAB, 2048, 50, 0.1, True, 300, False),
        # Chunks of six prompts marked in the counts of their slots: latency.
        _seen("seen_chunk", 16, 6, 400, VOCAB, False, 7),
        # Sixteen new prompts take their slots: counts cleared, prompts marked.
        _seen("seen_prompts", 32, 16, 4096, VOCAB, True, 9),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    kind = rng.choice(["rope", "append", "lora", "lora", "lora", "pick", "pick", "seen"])
    if kind in ("rope", "append"):
        hq, hkv, d = rng.choice([(16, 2, 128), (16, 8, 128), (14, 2, 64), (6, 3, 80), (4, 1, 256)])
        rot = rng.choice([d, d // 2])
        inter = rng.random() < 0.5
        if kind == "rope":
            return _rope("", _log(rng, 1, 12000), hq, d, rot, inter)
        q = _log(rng, 1, 4096)
        batch = _log(rng, 1, max(1, min(64, 12000 // q)))
        return _append("", batch, q, q + _log(rng, 1, 4096), hq, hkv, d, rng.choice([16, 32, 64, 128]), rot, inter,
                       rng.randrange(1, 10**6))
    if kind == "lora":
        k, columns = rng.choice([(2048, "2048+256+256"), (2048, "2048"), (2048, "11008+11008"), (11008, "2048"),
                                 (896, "896+128+128"), (1024, "2048+1024+1024"), (1024, "1000"), (256, "136+8")])
        n = sum(_widths(columns))
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        adapters = _log(rng, 1, max(1, min(64, 30_000_000 // (rank * (len(_widths(columns)) * k + n)))))
        none = rng.choice([0.0, 0.2])
        most = min(8192, 130_000_000 // (2 * k + 4 * n),
                   4_900_000_000 // (rank * (len(_widths(columns)) * k + n)))
        if rng.random() < 0.5:
            rows = _log(rng, 1, min(256, most))
            return _lora("", rows, rows, adapters, rank, k, columns, none, "rows")
        rows = _log(rng, 2, most)
        return _lora("", rows, _log(rng, 1, min(12, rows)), adapters, rank, k, columns, none, "sequences")
    if kind == "pick":
        k, n = rng.choice([(896, 1000), (1024, VOCAB), (2048, VOCAB), (2048, 32000), (1024, 5003)])
        rows = rng.randrange(1, 17)
        return _pick("", rows, n, k, rng.choice([1, 1, 5, 20, 50, 64]), rng.choice([0.01, 0.1, 0.4]),
                     rng.random() < 0.5, rng.choice([0, 4, 300]), rng.random() < 0.3)
    slots = _log(rng, 1, 64)
    return _seen("", slots, rng.randrange(1, min(slots, 16) + 1), _log(rng, 1, 8192), rng.choice([1000, 5003, VOCAB]),
                 rng.random() < 0.5, rng.randrange(1, 10**6))


def _widths(columns):
    return [int(c) for c in columns.split("+")]


def _lengths(case):
    """New tokens and tokens in the cache of each sequence: from a third to all of the new tokens, contexts spread
    over a factor of 16.  A function of the case alone."""
    n, q, ctx = case["batch"], case["q"], case["ctx"]
    rng = np.random.RandomState(case["ragged"])
    ql = rng.randint((q + 2) // 3, q + 1, n)
    kl = np.exp(rng.uniform(math.log(max(1.0, ctx / 16)), math.log(ctx), n)).astype(np.int64)
    ql[0], kl[0] = q, ctx
    return ql.astype(np.int64), np.maximum(kl, ql)


def _adapter_of_rows(case):
    """Adapter of every row, -1 for none: by row for decoding requests, by sequence for prompts.  A function of the
    case alone."""
    rng = np.random.RandomState(case["rows"] * 31 + case["rank"])
    n, count = case["rows"], case["sequences"]
    of_seq = rng.randint(0, case["adapters"], count)
    of_seq[rng.random_sample(count) < case["none"]] = -1
    if case["layout"] == "rows":
        return of_seq
    share = rng.random_sample(count) + 0.2
    ends = np.minimum(np.round(np.cumsum(share) / share.sum() * n), n).astype(np.int64)
    ends[-1] = n
    return np.repeat(of_seq, np.diff(np.concatenate([[0], ends])))


def _token_counts(case):
    """Tokens of each prompt: from a quarter of the longest to all of it."""
    rng = np.random.RandomState(case["ragged"])
    got = rng.randint((case["tokens"] + 3) // 4, case["tokens"] + 1, case["batch"])
    got[0] = case["tokens"]
    return got


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["hq"] * case["d"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 5 * n + 3 * case["tokens"] * case["hq"] * case["rot"]}
    if op == "append":
        tokens = int(_lengths(case)[0].sum())
        heads = case["hq"] + case["hkv"]
        return {"bytes": 4 * tokens * case["d"] * (heads + case["hkv"]) + 4 * tokens,
                "flops": tokens * heads * (5 * case["d"] + 3 * case["rot"])}
    if op == "lora":
        ids = _adapter_of_rows(case)
        widths, rank, k = _widths(case["columns"]), case["rank"], case["k"]
        n, used = sum(widths), len(set(ids[ids >= 0].tolist()))
        with_one = int((ids >= 0).sum())
        return {"bytes": 2 * with_one * k + 4 * len(ids) * n + 2 * used * rank * (len(widths) * k + n),
                "flops": 2 * with_one * rank * (len(widths) * k + n)}
    if op == "pick":
        rows, n, k = case["rows"], case["n"], case["k"]
        weight = n * k // 2 + (n * k // 128 * 2 if case["symmetric"] else n * k // 64 * 4)
        return {"bytes": weight + 2 * rows * k + 2 * rows * n + (rows * n // 8 if case["masked"] else 0) +
                8 * rows * case["biases"] + 8 * rows * case["top"], "flops": 2 * rows * n * k}
    tokens = int(_token_counts(case).sum())
    return {"bytes": 4 * tokens + (2 * case["batch"] * case["n"] if case["reset"] else 4 * tokens), "flops": tokens}


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _head_inputs(case, seed):
    gen = _gen(seed)
    hq, d = case["hq"], case["d"]
    turns = np.round(_theta(case) / (2.0 * math.pi) * 2.0**64).astype(np.uint64).view(np.int64)
    s = {"case": case, "turns": torch.from_numpy(turns).to(DEVICE)}
    # Before the norm, heads differ in size by a factor of 30, and a few elements stand out.
    size = torch.exp2(torch.linspace(-3.0, 2.0, hq, device=DEVICE))[:, None]
    out = 1.0 + 7.0 * (torch.arange(d, device=DEVICE) % 37 == 5)
    s["q_weight"] = 1.0 + 0.3 * _normal(gen, d)
    if case["op"] == "rope":
        t = case["tokens"]
        s["x"] = (_normal(gen, t, hq, d) * size * out).half()
        start = torch.randint(0, 4096, (1,), generator=gen, device=DEVICE)
        s["positions"] = (start + torch.arange(t, device=DEVICE)).to(torch.int32)
        s["y"] = torch.empty_like(s["x"])
        return s
    ql, kl = _lengths(case)
    n, page, hkv, tokens = case["batch"], case["page"], case["hkv"], int(ql.sum())
    need = -(-kl // page)
    pages = int(need.sum()) + 3
    order = np.random.RandomState(seed % 2**32).permutation(pages)
    table = np.full((n, int(need.max())), -1, np.int32)
    first = np.cumsum(need) - need
    b_of_page = np.repeat(np.arange(n), need)
    table[b_of_page, np.arange(need.sum()) - first[b_of_page]] = order[:need.sum()]
    offsets = np.concatenate([[0], np.cumsum(ql)])
    b_of = np.repeat(np.arange(n), ql)
    i_of = np.arange(tokens) - offsets[b_of]
    s["table"] = torch.from_numpy(table).to(DEVICE)
    s["q_offsets"] = torch.from_numpy(offsets.astype(np.int32)).to(DEVICE)
    s["kv_lens"] = torch.from_numpy(kl.astype(np.int32)).to(DEVICE)
    s["b_of"], s["i_of"] = torch.from_numpy(b_of).to(DEVICE), torch.from_numpy(i_of).to(DEVICE)
    s["tokens"], s["max_q"] = tokens, int(ql.max())
    # One projection's output: the heads of q, k and v of a token side by side.
    qkv = _normal(gen, tokens, hq + 2 * hkv, d)
    qkv[:, :hq] *= size
    qkv[:, :hq + hkv] *= out
    s["qkv"] = qkv.half()
    s["k_weight"] = 1.0 + 0.3 * _normal(gen, d)
    s["k_cache"] = _normal(gen, pages, page, hkv, d).half()
    s["v_cache"] = _normal(gen, pages, page, hkv, d).half()
    s["y"] = torch.empty(tokens, hq, d, device=DEVICE, dtype=torch.float16)
    return s


def _lora_inputs(case, seed):
    gen = _gen(seed)
    widths, rank, k, m = _widths(case["columns"]), case["rank"], case["k"], case["rows"]
    n, count = sum(widths), case["adapters"]
    ids = _adapter_of_rows(case)
    s = {"case": case, "widths": widths, "ids_host": ids}
    s["x"] = _normal(gen, m, k).half()
    s["y"] = _normal(gen, m, n).half()
    s["a"] = (_normal(gen, count, len(widths), rank, k) * k**-0.5).half()
    s["b"] = (_normal(gen, count, n, rank) * 0.05).half()
    s["scale"] = torch.exp2(torch.randint(-1, 3, (count,), generator=gen, device=DEVICE).float()) * 0.9
    s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(DEVICE)
    s["out"] = torch.empty_like(s["y"])
    return s


def _pick_inputs(case, seed):
    """Weights and activations on coarse grids: every sum of products is exact in 32 bits in any order, so that the
    order of the logits, and with it the selection, is defined; equal logits go to the lowest index."""
    gen = _gen(seed)
    m, n, k, top = case["rows"], case["n"], case["k"], case["top"]
    group = 128 if case["symmetric"] else 64
    s = {"case": case, "group": group}
    s["x"] = (_normal(gen, m, k) * 8.0).round_().clamp_(-32.0, 32.0).div_(8.0).half()
    s["qweight"] = torch.randint(-2**31, 2**31, (n, k // 8), generator=gen, device=DEVICE, dtype=torch.int32)
    steps = torch.randint(4, 41, (n, k // group), generator=gen, device=DEVICE).float()  # scales of 0.002 to 0.02
    s["scales"] = (steps * 2.0**-11).half()
    s["biases"] = None
    if not case["symmetric"]:
        around = torch.randint(-2, 3, steps.shape, generator=gen, device=DEVICE).float()
        s["biases"] = ((around - 8.0 * steps) * 2.0**-11).half()
    # Requests sit in any slots of the counts.
    slots = m + 3
    s["slots"] = torch.randperm(slots, generator=gen, device=DEVICE)[:m].to(torch.int32)
    seen = torch.rand(slots, n, generator=gen, device=DEVICE) < case["seen"]
    times = torch.randint(0, 5, (slots, n), generator=gen, device=DEVICE)  # in the output; 0: in the prompt alone
    prompt = (torch.rand(slots, n, generator=gen, device=DEVICE) < 0.5) | (times == 0)
    s["counts"] = torch.where(seen, times + prompt * PROMPT, torch.zeros_like(times)).to(torch.int16)
    s["repetition"] = 1.0 + 0.05 * torch.randint(0, 8, (m,), generator=gen, device=DEVICE).float()
    s["presence"] = 0.125 * torch.randint(0, 5, (m,), generator=gen, device=DEVICE).float()
    s["frequency"] = 0.1 * torch.randint(0, 5, (m,), generator=gen, device=DEVICE).float()
    s["bias_offsets"] = s["allowed"] = None
    if case["biases"]:
        per = case["biases"]
        s["bias_offsets"] = (torch.arange(m + 1, device=DEVICE) * per).to(torch.int32)
        s["bias_tokens"] = torch.cat([torch.randperm(n, generator=gen, device=DEVICE)[:per]
                                      for _ in range(m)]).to(torch.int32)
        s["bias_values"] = 0.25 * torch.randint(-40, 41, (m * per,), generator=gen, device=DEVICE).float()
    if case["masked"]:
        # Everything, about half, or a handful of the vocabulary; the last of several rows is left nothing.
        share = torch.tensor([1.0, 0.5, 20.0 / n, 0.05], device=DEVICE)[torch.arange(m, device=DEVICE) % 4]
        allowed = torch.rand(m, (n + 31) // 32 * 32, generator=gen, device=DEVICE) < share[:, None]
        if m > 4:
            allowed[m - 1] = False
        bits = allowed.view(m, -1, 32).long() << torch.arange(32, device=DEVICE)
        s["allowed_bools"] = allowed[:, :n]
        s["allowed"] = bits.sum(-1).to(torch.int32)
    s["idx"] = torch.empty(m, top, device=DEVICE, dtype=torch.int32)
    s["val"] = torch.empty(m, top, device=DEVICE, dtype=torch.float32)
    return s


def _seen_inputs(case, seed):
    gen = _gen(seed)
    n, batch = case["n"], case["batch"]
    lens = _token_counts(case)
    s = {"case": case, "total": int(lens.sum())}
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).to(DEVICE)
    s["b_of"] = torch.from_numpy(np.repeat(np.arange(batch), lens)).to(DEVICE)
    # Few tokens are frequent, most are rare.
    u = torch.rand(s["total"], generator=gen, device=DEVICE)
    s["tokens"] = (n ** u - 1.0).long().clamp(0, n - 1).to(torch.int32)
    s["slots"] = torch.randperm(case["slots"], generator=gen, device=DEVICE)[:batch].to(torch.int32)
    s["counts"] = torch.randint(0, 3, (case["slots"], n), generator=gen, device=DEVICE, dtype=torch.int16)
    return s


def _inputs(case, seed):
    return {"rope": _head_inputs, "append": _head_inputs, "lora": _lora_inputs, "pick": _pick_inputs,
            "seen": _seen_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import int4_weight_only_affine_gb300 as w4
        s["w4"] = w4
        op = case["op"]
        if op in ("rope", "append"):
            s["rope"] = w4.Rope(s["turns"], interleaved=case["interleaved"])
            s["q_norm"] = w4.HeadNorm(s["q_weight"], EPS)
        if op == "append":
            s["k_norm"] = w4.HeadNorm(s["k_weight"], EPS)
            s["cache"] = w4.KVCache(s["k_cache"], s["v_cache"])
            s["batch"] = w4.KVBatch(s["table"], s["q_offsets"], s["kv_lens"], s["tokens"], s["max_q"])
        if op == "lora":
            s["set"] = w4.Adapters(s["a"], s["b"], scale=s["scale"], columns=s["widths"])
        if op in ("pick", "seen"):
            s["table"] = w4.TokenCounts(s["counts"])
        if op == "pick":
            biases = None if s["bias_offsets"] is None else (s["bias_offsets"], s["bias_tokens"], s["bias_values"])
            s["rules"] = w4.LogitRules(counts=s["table"], slots=s["slots"], repetition=s["repetition"],
                                       presence=s["presence"], frequency=s["frequency"], biases=biases,
                                       allowed=s["allowed"])
            need = w4.lm_head_workspace_bytes(case["rows"], case["n"], case["top"])
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEVICE)
    return s


# ----------------------------------------------------------- the plain forms

def _theta(case):
    """Angle per position of each rotated pair, in radians (64 bits)."""
    i = np.arange(case["rot"] // 2, dtype=np.float64)
    return BASE ** (-2.0 * i / case["rot"])


def _cos_sin(s, positions):
    """float32 [tokens][rot / 2]: the angle as a fraction of a turn, exact in wrapping 64-bit integers."""
    fraction = positions.long()[:, None] * s["turns"]
    angle = fraction.double().mul_(2.0**-64).float() * (2.0 * math.pi)
    return torch.cos(angle), torch.sin(angle)


def _norm_rotate(x, weight, cos, sin, interleaved):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1).half()


def _append_plain(s):
    c = s["case"]
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    lens = s["q_offsets"][1:] - s["q_offsets"][:-1]
    p = (s["kv_lens"] - lens)[s["b_of"]] + s["i_of"]
    cos, sin = _cos_sin(s, p)
    where = s["table"][s["b_of"], p // page].long()
    q, k, v = s["qkv"].split([hq, hkv, hkv], 1)
    s["k_cache"][where, p % page] = _norm_rotate(k, s["k_weight"], cos, sin, c["interleaved"])
    s["v_cache"][where, p % page] = v
    return {"q": _norm_rotate(q, s["q_weight"], cos, sin, c["interleaved"]), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _spans(ids):
    """(first, end, adapter) of each run of rows of one adapter."""
    cut = np.flatnonzero(np.diff(ids)) + 1
    return [(int(a), int(b), int(ids[a])) for a, b in zip(np.r_[0, cut], np.r_[cut, len(ids)])]


def _lora_plain(s):
    c, widths, rank = s["case"], s["widths"], s["case"]["rank"]
    if c["layout"] == "rows":  # every row's own adapter, gathered
        at = s["ids"].clamp(min=0).long()
        h = torch.einsum("mk,msrk->msr", s["x"].float(), s["a"][at].float())
        h = h * torch.where(s["ids"] >= 0, s["scale"][at], torch.zeros_like(s["scale"][at]))[:, None, None]
        parts = [torch.einsum("mr,mnr->mn", h[:, i], b.float()) for i, b in enumerate(s["b"][at].split(widths, 1))]
        return {"out": (s["y"].float() + torch.cat(parts, 1)).half()}
    out = s["y"].float()
    for first, end, adapter in _spans(s["ids_host"]):
        if adapter < 0:
            continue
        x = s["x"][first:end].float()
        col = 0
        for i, w in enumerate(widths):
            h = x @ s["a"][adapter, i].float().T * s["scale"][adapter]
            out[first:end, col:col + w] += h @ s["b"][adapter, col:col + w].float().T
            col += w
    return {"out": out.half()}


def _codes(s):
    shifts = torch.arange(0, 32, 4, device=DEVICE, dtype=torch.int32)
    return ((s["qweight"][:, :, None] >> shifts) & 15).flatten(1)


def _weights(s, dtype):
    n = s["qweight"].shape[0]
    q = _codes(s).view(n, -1, s["group"]).to(dtype)
    scale = s["scales"].to(dtype)[:, :, None]
    return (scale * q + s["biases"].to(dtype)[:, :, None] if s["biases"] is not None else scale * (q - 8.0)).view(n, -1)


def _pick_plain(s):
    c = s["case"]
    m, top = c["rows"], c["top"]
    z = s["x"].float() @ _weights(s, torch.float32).T
    counts = s["counts"][s["slots"].long()].int() & 0xFFFF
    seen, times = counts != 0, (counts & 0x7FFF).float()
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * times
    z = torch.where(times > 0, z - s["presence"][:, None], z)
    if s["bias_offsets"] is not None:
        row = torch.arange(m, device=DEVICE).repeat_interleave(c["biases"])
        z = z.index_put((row, s["bias_tokens"].long()), s["bias_values"], accumulate=True)
    if s["allowed"] is not None:
        z = z.masked_fill(~s["allowed_bools"], -math.inf)
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)  # equal values: the lowest index first
    val, idx = val[:, :top].contiguous(), idx[:, :top].to(torch.int32)
    return {"idx": idx.masked_fill(val == -math.inf, -1), "val": val}


def _seen_plain(s):
    c = s["case"]
    at = s["slots"].long()
    if c["reset"]:
        s["counts"][at] = 0
    rows, tokens = at[s["b_of"]], s["tokens"].long()
    s["counts"][rows, tokens] = s["counts"][rows, tokens] | -PROMPT  # (the same value however often a token comes)
    return {"counts": s["counts"]}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "rope":
            return {"y": _norm_rotate(s["x"], s["q_weight"], *_cos_sin(s, s["positions"]), c["interleaved"])}
        return {"append": _append_plain, "lora": _lora_plain, "pick": _pick_plain, "seen": _seen_plain}[op](s)
    w4 = s["w4"]
    if op == "rope":
        return {"y": w4.f16_rope(s["x"], s["rope"], s["positions"], y=s["y"], norm=s["q_norm"])}
    if op == "append":
        hq, hkv, qkv = c["hq"], c["hkv"], s["qkv"]
        q = w4.f16_kv_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], s["cache"], s["batch"], rope=s["rope"],
                             q=qkv[:, :hq], y=s["y"], q_norm=s["q_norm"], k_norm=s["k_norm"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "lora":
        return {"out": w4.f16_lora(s["x"], s["set"], s["ids"], s["y"], out=s["out"])}
    if op == "pick":
        idx, val = w4.lm_head_argmax_topk(s["x"], s["qweight"], s["scales"], s["biases"], k=c["top"], idx=s["idx"],
                                          val=s["val"], workspace=s["workspace"], group=s["group"], rules=s["rules"])
        return {"idx": idx, "val": val}
    w4.token_counts_add(s["table"], s["slots"], s["tokens"], offsets=s["offsets"], prompt=True, reset=c["reset"])
    return {"counts": s["counts"]}


# ------------------------------------------------------ the definitions in 64 bits

def _normed_turned(case, x, weight, positions):
    """x [tokens][heads][d], normed and rotated by the definition, in complex numbers."""
    x = x.double()
    x = x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / x.shape[-1] + EPS) * weight.double()
    half = case["rot"] // 2
    angle = positions.double()[:, None] * torch.from_numpy(_theta(case)).to(DEVICE)
    wheel = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    even = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
    odd = even + (1 if case["interleaved"] else half)
    z = torch.complex(x[..., even], x[..., odd]) * wheel
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _append_exact(case, s):
    ql, kl = _lengths(case)
    hq, hkv, page = case["hq"], case["hkv"], case["page"]
    table = s["table"].cpu().numpy().astype(np.int64)
    where, positions = [], []
    for b in range(len(ql)):
        p = np.arange(kl[b] - ql[b], kl[b])
        where.append(table[b, p // page] * page + p % page)
        positions.append(p)
    where = torch.from_numpy(np.concatenate(where)).to(DEVICE)
    p = torch.from_numpy(np.concatenate(positions)).to(DEVICE)
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k.flatten(0, 1)[where] = _normed_turned(case, s["qkv"][:, hq:hq + hkv], s["k_weight"], p)
    v.flatten(0, 1)[where] = s["qkv"][:, hq + hkv:].double()
    return {"q": _normed_turned(case, s["qkv"][:, :hq], s["q_weight"], p), "k_cache": k, "v_cache": v}


def _lora_exact(case, s):
    out = s["y"].double()
    ids = s["ids_host"]
    edges = np.cumsum([0] + s["widths"])
    for adapter in sorted(set(ids[ids >= 0].tolist())):
        rows = torch.from_numpy(np.flatnonzero(ids == adapter)).to(DEVICE)
        x = s["x"][rows].double()
        for i in range(len(s["widths"])):
            delta = (s["b"][adapter, edges[i]:edges[i + 1]].double() @ (s["a"][adapter, i].double() @ x.T)).T
            out[rows, edges[i]:edges[i + 1]] += float(s["scale"][adapter]) * delta
    return {"out": out}


def _pick_exact(case, s):
    m, n, top = case["rows"], case["n"], case["top"]
    logits = torch.cat([s["x"].double() @ _weights({**s, **{key: None if s[key] is None else s[key][r:r + 8192]
                                                            for key in ("qweight", "scales", "biases")}},
                                                   torch.float64).T for r in range(0, n, 8192)], 1).cpu().numpy()
    counts, slots = s["counts"].cpu().numpy().view(np.uint16), s["slots"].cpu().numpy()
    par = {key: s[key].double().cpu().numpy() for key in ("repetition", "presence", "frequency")}
    idx, val = np.full((m, top), -1, np.int32), np.full((m, top), -np.inf)
    for r in range(m):
        z, c = logits[r].copy(), counts[slots[r]]
        up, down = (c > 0) & (z > 0), (c > 0) & (z <= 0)
        z[up] /= par["repetition"][r]
        z[down] *= par["repetition"][r]
        times = c % PROMPT
        z -= par["frequency"][r] * times + par["presence"][r] * (times > 0)
        if s["bias_offsets"] is not None:
            lo, hi = s["bias_offsets"][r:r + 2].tolist()
            np.add.at(z, s["bias_tokens"][lo:hi].cpu().numpy(), s["bias_values"][lo:hi].double().cpu().numpy())
        left = np.arange(n) if s["allowed"] is None else np.flatnonzero(s["allowed_bools"][r].cpu().numpy())
        best = left[np.lexsort((left, -z[left]))[:top]]
        idx[r, :len(best)], val[r, :len(best)] = best, z[best]
    return {"idx": torch.from_numpy(idx), "val": torch.from_numpy(val)}


def _seen_exact(case, s):
    counts = s["counts"].cpu().numpy().view(np.uint16).copy()
    offsets, tokens = s["offsets"].tolist(), s["tokens"].cpu().numpy()
    for b, slot in enumerate(s["slots"].tolist()):
        if case["reset"]:
            counts[slot] = 0
        mine = np.unique(tokens[offsets[b]:offsets[b + 1]])
        counts[slot, mine] |= np.uint16(PROMPT)
    return {"counts": torch.from_numpy(counts.view(np.int16))}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        return {"y": _normed_turned(case, s["x"], s["q_weight"], s["positions"])}
    return {"append": _append_exact, "lora": _lora_exact, "pick": _pick_exact, "seen": _seen_exact}[op](case, s)
