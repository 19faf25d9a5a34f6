"""Cases of the attention operators, with their plain forms.

Three operators of a transformer layer between its projections: rotary
positions (f16_rope), keys and values appended to a paged cache with the
rotation applied on the way (f16_kv_append), and attention of a chunk of new
tokens over that cache (f16_attention).  With own = False run() computes them
with elementary torch operations in 32 bits, with own = True by the
framework's calls.  exact() restates the definitions in 64 bits.

Sequences: sequence b brings q_len[b] new tokens and has kv_len[b] tokens in
the cache after they are appended; its token i stands at position
kv_len - q_len + i.  Token positions map to cache slots through a table of
pages per sequence.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
BASE = 1000000.0  # base of the rotation's wavelengths (long-context setting)


# ---------------------------------------------------------------- the cases

def _rope(name, tokens, heads, d, rot, interleaved, stretch):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": heads, "d": d, "rot": rot,
            "interleaved": interleaved, "stretch": stretch}


def _append(name, batch, q, ctx, hq, hkv, d, page, rot, interleaved, ragged):
    return {"name": name, "op": "append", "batch": batch, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "rot": rot, "interleaved": interleaved, "ragged": ragged, "mixed": False, "stretch": 1.0}


def _attend(name, batch, q, ctx, hq, hkv, d, page, ragged, mixed=False, window=0, lse=False):
    return {"name": name, "op": "attend", "batch": batch, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "ragged": ragged, "mixed": mixed, "window": window, "lse": lse}


def listed():
    return [
        # Queries of one decode step of eight sequences (16 heads of 128): latency.
        _rope("rope_step", 8, 16, 128, 128, False, 1.0),
        # Queries of a long prompt, half of each head rotated, positions stretched four times: bandwidth.
        _rope("rope_prompt", 16384, 16, 128, 64, True, 4.0),
        # One decode step of 16 sequences, 16 query and 2 key/value heads of 128: latency.
        _append("append_step", 16, 1, 2000, 16, 2, 128, 16, 128, False, 3),
        # Chunks of six prompts, 14 query and 2 key/value heads of 64.
        _append("append_chunks", 6, 400, 1500, 14, 2, 64, 64, 64, False, 5),
        # Four prompts of 4096 tokens, 16 query and 8 key/value heads of 128: bandwidth.
        _append("append_prompts", 4, 4096, 4096, 16, 8, 128, 64, 128, True, 0),
        # One sequence's decode step over a short context: latency.
        _attend("attend_step", 1, 1, 600, 16, 2, 128, 16, 0),
        # Decode step of a full batch over contexts of very different lengths, one slot of the batch empty.
        _attend("attend_batch", 48, 1, 8192, 16, 8, 128, 16, 7, lse=True),
        # One sequence's decode step over a long context: bandwidth on few rows.
        _attend("attend_long", 1, 1, 131071, 16, 2, 128, 64, 0),
        # A short chunk (a few prompt tokens, or drafted ones) over a long context.
        _attend("attend_chunk", 1, 64, 16001, 16, 8, 128, 32, 0, lse=True),
        # Decode steps and prompt chunks in one batch, sliding window, heads of 64.
        _attend("attend_mixed", 9, 500, 4000, 14, 2, 64, 16, 11, mixed=True, window=1024),
        # A prompt of 1570 tokens into an empty cache.
        _attend("attend_prompt", 1, 1570, 1570, 16, 2, 128, 16, 0),
        # A long prompt into an empty cache: arithmetic.
        _attend("attend_prompt_long", 1, 8192, 8192, 16, 8, 128, 64, 0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    hq, hkv, d = rng.choice([(16, 2, 128), (16, 8, 128), (14, 2, 64)])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.randrange(1, 10**6)
    inter = rng.random() < 0.5
    rot = rng.choice([d, d // 2])
    kind = rng.choice(["rope", "append", "step", "step", "chunk", "prompt"])
    if kind == "rope":
        return _rope("", _log(rng, 1, 16384), hq, d, rot, inter, rng.choice([1.0, 2.0, 4.0]))
    if kind == "append":
        q = _log(rng, 1, 4096)
        batch = _log(rng, 1, max(1, min(64, 16384 // q)))
        return _append("", batch, q, q + _log(rng, 1, 4096), hq, hkv, d, page, rot, inter, ragged)
    if kind == "step":
        ctx = _log(rng, 1, 131072)
        batch = _log(rng, 1, max(1, min(64, 262144 // ctx)))
        return _attend("", batch, 1, ctx, hq, hkv, d, page, ragged, lse=rng.random() < 0.5)
    window = rng.choice([0, 0, 1024])
    if kind == "chunk":
        q = _log(rng, 2, 512)
        ctx = q + _log(rng, 1, 16384)
        batch = _log(rng, 1, max(1, min(8, 2**23 // (q * ctx))))
        return _attend("", batch, q, ctx, hq, hkv, d, page, ragged, rng.random() < 0.5, window, rng.random() < 0.5)
    q = _log(rng, 256, 8192)
    batch = _log(rng, 1, max(1, min(8, 2**25 // (q * q))))
    return _attend("", batch, q, q, hq, hkv, d, page, ragged, False, window, rng.random() < 0.5)


def _lengths(case):
    """New tokens and tokens in the cache of each sequence: a function of the case alone.

    ragged: from a third to all of the new tokens, and contexts spread over a
    factor of 16; a batch of single tokens has one empty slot (no tokens in
    the cache), as a padded batch has.  mixed: all but every fourth sequence
    bring one token."""
    n, q, ctx = case["batch"], case["q"], case["ctx"]
    if not case["ragged"]:
        return np.full(n, q, np.int64), np.full(n, ctx, np.int64)
    rng = np.random.RandomState(case["ragged"])
    ql = rng.randint((q + 2) // 3, q + 1, n)
    kl = np.exp(rng.uniform(math.log(max(1.0, ctx / 16)), math.log(ctx), n)).astype(np.int64)
    if case["mixed"]:
        ql[np.arange(n) % 4 != 0] = 1
    ql[0], kl[0] = q, ctx
    kl = np.maximum(kl, ql)
    if case["op"] == "attend" and q == 1 and n > 8:
        kl[n // 2] = 0
    return ql.astype(np.int64), kl


def _theta(case):
    """Angle per position of each rotated pair, in radians (64 bits)."""
    i = np.arange(case["rot"] // 2, dtype=np.float64)
    return BASE ** (-2.0 * i / case["rot"]) / case["stretch"]


def _factor(case):
    """Scale of rotated values of a stretched context."""
    return 0.1 * math.log(case["stretch"]) + 1.0


def work(case):
    hq, d = case["hq"], case["d"]
    if case["op"] == "rope":
        n = case["tokens"] * hq * d
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * case["tokens"] * hq * case["rot"]}
    ql, kl = _lengths(case)
    tokens, hkv = int(ql.sum()), case["hkv"]
    if case["op"] == "append":
        return {"bytes": 4 * tokens * d * (hq + 2 * hkv) + 4 * tokens, "flops": 3 * tokens * (hq + hkv) * case["rot"]}
    pairs = seen = 0
    for q, k in zip(ql.tolist(), kl.tolist()):
        last = np.minimum(np.arange(k - q, k) + 1, k).clip(min=0)  # keys up to the row's own
        first = (np.arange(k - q, k) - case["window"] + 1).clip(min=0) if case["window"] else 0 * last
        pairs += int((last - first).clip(min=0).sum())
        seen += int(max(0, last.max() - first.min())) if q else 0
    size = 4 * tokens * hq * d + 4 * hkv * d * seen + 4 * seen // case["page"] + (4 * tokens * hq if case["lse"] else 0)
    return {"bytes": size, "flops": 4 * d * hq * pairs}


# --------------------------------------------------------------- the inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32).half()


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    hq, d = case["hq"], case["d"]
    s = {"case": case}
    if case["op"] != "attend":
        turns = np.round(_theta(case) / (2.0 * math.pi) * 2.0**64).astype(np.uint64).view(np.int64)
        s["turns"] = torch.from_numpy(turns).to(DEVICE)
        s["factor"] = _factor(case)
    if case["op"] == "rope":
        t = case["tokens"]
        s["x"] = _normal(gen, t, hq, d)
        # positions of a prompt's tokens, or of a step's sequences anywhere in a long context
        start = torch.randint(0, 4096, (1,), generator=gen, device=DEVICE)
        s["positions"] = (torch.randint(0, 131072, (t,), generator=gen, device=DEVICE) if t <= 64
                          else start + torch.arange(t, device=DEVICE)).to(torch.int32)
        s["y"] = torch.empty_like(s["x"])
        return s
    ql, kl = _lengths(case)
    n, page, hkv, tokens = case["batch"], case["page"], case["hkv"], int(ql.sum())
    need = -(-kl // page)
    pages = int(need.sum()) + 3
    order = np.random.RandomState(seed % 2**32).permutation(pages)
    table = np.full((n, max(1, int(need.max()))), -1, np.int32)
    start = np.cumsum(need) - need
    b_of_page = np.repeat(np.arange(n), need)
    table[b_of_page, np.arange(need.sum()) - start[b_of_page]] = order[:need.sum()]
    offsets = np.concatenate([[0], np.cumsum(ql)])
    b_of = np.repeat(np.arange(n), ql)
    i_of = np.arange(tokens) - offsets[b_of]
    s["table"] = torch.from_numpy(table).to(DEVICE)
    s["q_offsets"] = torch.from_numpy(offsets.astype(np.int32)).to(DEVICE)
    s["kv_lens"] = torch.from_numpy(kl.astype(np.int32)).to(DEVICE)
    s["b_of"], s["i_of"] = torch.from_numpy(b_of).to(DEVICE), torch.from_numpy(i_of).to(DEVICE)
    s["tokens"], s["max_q"] = tokens, int(ql.max())
    # Heads differ in how sharply they attend, and the first token of a sequence draws weight.
    sharp = torch.exp2(torch.linspace(-1.0, 1.5, hq, device=DEVICE))
    s["q"] = (torch.randn(tokens, hq, d, generator=gen, device=DEVICE) + 0.3).mul_(sharp[:, None]).half()
    s["k_cache"] = _normal(gen, pages, page, hkv, d)
    s["v_cache"] = _normal(gen, pages, page, hkv, d)
    first = table[:, 0][need > 0].astype(np.int64)
    s["k_cache"][torch.from_numpy(first).to(DEVICE), 0] += 0.2
    s["y"] = torch.empty_like(s["q"])
    if case["op"] == "append":
        s["k"], s["v"] = _normal(gen, tokens, hkv, d), _normal(gen, tokens, hkv, d)
    elif case["lse"]:
        s["lse"] = torch.empty(tokens, hq, device=DEVICE, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import int4_weight_only_affine_gb300 as w4
        s["w4"] = w4
        if "turns" in s:
            s["rope"] = w4.Rope(s["turns"], interleaved=case["interleaved"], factor=s["factor"])
        if case["op"] != "rope":
            s["cache"] = w4.KVCache(s["k_cache"], s["v_cache"])
            s["batch"] = w4.KVBatch(s["table"], s["q_offsets"], s["kv_lens"], s["tokens"], s["max_q"])
        if case["op"] == "attend":
            s["workspace"] = w4.attention_workspace(s["cache"], case["hq"], s["max_q"])
    return s


# ----------------------------------------------------------- the plain forms

def _cos_sin(s, positions):
    """float32 [tokens][rot / 2]: the angle as a fraction of a turn, exact in wrapping 64-bit integers."""
    fraction = positions.long()[:, None] * s["turns"]
    angle = fraction.double().mul_(2.0**-64).float() * (2.0 * math.pi)
    return torch.cos(angle) * s["factor"], torch.sin(angle) * s["factor"]


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[1]
    x = x.float()
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1).half()


def _positions(s):
    lens = s["q_offsets"][1:] - s["q_offsets"][:-1]
    return (s["kv_lens"] - lens)[s["b_of"]] + s["i_of"]


def _append_plain(s):
    page = s["case"]["page"]
    p = _positions(s)
    cos, sin = _cos_sin(s, p)
    where = s["table"][s["b_of"], p // page].long()
    s["k_cache"][where, p % page] = _rotate(s["k"], cos, sin, s["case"]["interleaved"])
    s["v_cache"][where, p % page] = s["v"]
    return {"q": _rotate(s["q"], cos, sin, s["case"]["interleaved"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend_plain(s):
    c = s["case"]
    n, hkv, d, group, width = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"], s["max_q"]
    table = s["table"].clamp(min=0).long()
    k = s["k_cache"][table].flatten(1, 2).permute(0, 2, 3, 1).float()  # [n][hkv][d][keys]
    v = s["v_cache"][table].flatten(1, 2).transpose(1, 2).float()  # [n][hkv][keys][d]
    q = torch.zeros(n, width, hkv, group, d, device=DEVICE)
    q[s["b_of"], s["i_of"]] = s["q"].float().view(-1, hkv, group, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, group * width, d)
    scores = torch.matmul(q, k).view(n, hkv, group, width, -1).mul_(d**-0.5)
    lens = s["q_offsets"][1:] - s["q_offsets"][:-1]
    own_key = (s["kv_lens"] - lens)[:, None, None] + torch.arange(width, device=DEVICE)[:, None]
    key = torch.arange(scores.shape[-1], device=DEVICE)
    seen = (key <= own_key) & (key < s["kv_lens"][:, None, None])
    if c["window"]:
        seen &= key > own_key - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    y = torch.matmul(p.view(n, hkv, group * width, -1), v).view(n, hkv, group, width, d) / total.clamp(min=1e-30)
    out = {"y": y.permute(0, 3, 1, 2, 4)[s["b_of"], s["i_of"]].reshape(-1, c["hq"], d).half()}
    if c["lse"]:
        out["lse"] = (top + total.log()).permute(0, 3, 1, 2, 4)[s["b_of"], s["i_of"]].reshape(-1, c["hq"])
    return out


def run(s):
    c = s["case"]
    if own:
        w4 = s["w4"]
        if c["op"] == "rope":
            return {"y": w4.f16_rope(s["x"], s["rope"], s["positions"], y=s["y"])}
        if c["op"] == "append":
            q = w4.f16_kv_append(s["k"], s["v"], s["cache"], s["batch"], rope=s["rope"], q=s["q"], y=s["y"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        y = w4.f16_attention(s["q"], s["cache"], s["batch"], y=s["y"], lse=s.get("lse"), window=c["window"],
                             workspace=s["workspace"])
        return {"y": y, "lse": s["lse"]} if c["lse"] else {"y": y}
    if c["op"] == "rope":
        return {"y": _rotate(s["x"], *_cos_sin(s, s["positions"]), c["interleaved"])}
    return _append_plain(s) if c["op"] == "append" else _attend_plain(s)


# ------------------------------------------------------ the definitions in 64 bits

def _turned(case, x, positions):
    """x [tokens][heads][d] rotated by the definition, in complex numbers."""
    x = x.double()
    half = case["rot"] // 2
    angle = positions.double()[:, None] * torch.from_numpy(_theta(case)).to(DEVICE)
    wheel = torch.polar(torch.full_like(angle, _factor(case)), angle)[:, None, :]
    even = torch.arange(half, device=DEVICE) * (2 if case["interleaved"] else 1)
    odd = even + (1 if case["interleaved"] else half)
    z = torch.complex(x[..., even], x[..., odd]) * wheel
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return {"y": _turned(case, s["x"], s["positions"])}
    ql, kl = _lengths(case)
    at = np.cumsum(ql) - ql
    page, hkv, d, group = case["page"], case["hkv"], case["d"], case["hq"] // case["hkv"]
    table = s["table"].cpu().numpy()

    def slots(b, first, last):
        p = np.arange(first, last)
        return torch.from_numpy(table[b, p // page].astype(np.int64) * page + p % page).to(DEVICE)

    if case["op"] == "append":
        where = torch.cat([slots(b, kl[b] - ql[b], kl[b]) for b in range(len(ql))])
        p = torch.from_numpy(np.concatenate([np.arange(k - q, k) for q, k in zip(ql, kl)])).to(DEVICE)
        k_all, v_all = s["k_cache"].double().flatten(0, 1), s["v_cache"].double().flatten(0, 1)
        k_all[where], v_all[where] = _turned(case, s["k"], p), s["v"].double()
        return {"q": _turned(case, s["q"], p), "k_cache": k_all.view(s["k_cache"].shape),
                "v_cache": v_all.view(s["v_cache"].shape)}
    y = torch.zeros(s["tokens"], case["hq"], d, dtype=torch.float64, device=DEVICE)
    lse = torch.full((s["tokens"], case["hq"]), -math.inf, dtype=torch.float64, device=DEVICE)
    keys, values = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    for b in range(len(ql)):
        for r in range(0, int(ql[b]), 1024):  # rows r..e of the sequence, the keys that any of them sees
            e = min(int(ql[b]), r + 1024)
            p = np.arange(kl[b] - ql[b] + r, kl[b] - ql[b] + e)
            low = max(0, int(p[0]) - case["window"] + 1) if case["window"] else 0
            high = min(int(p[-1]) + 1, int(kl[b]))
            if high <= low:
                continue
            j, i = torch.arange(low, high, device=DEVICE), torch.from_numpy(p).to(DEVICE)
            hidden = j[None] > i[:, None]
            if case["window"]:
                hidden |= j[None] <= i[:, None] - case["window"]
            where = slots(b, low, high)
            rows = slice(int(at[b]) + r, int(at[b]) + e)
            for h in range(case["hq"]):
                z = s["q"][rows, h].double() @ keys[where, h // group].double().T / math.sqrt(d)
                z[hidden] = -math.inf
                lse[rows, h] = torch.logsumexp(z, 1)
                y[rows, h] = torch.softmax(z, 1) @ values[where, h // group].double()
    return {"y": y, "lse": lse} if case["lse"] else {"y": y}
