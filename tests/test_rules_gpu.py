"""Selection under rules (lm_head_argmax_topk with LogitRules) and token counts, exactly.

Weights and activations lie on coarse grids (x in eighths up to 4, scales and
biases in 2**-11): every sum of products is exact in fp32 in any order, so the
logits are known bit for bit, and so is each rule's fp32 step after them."""
import numpy as np
import pytest

from _gpu import require_gpu, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    yield w4
    assert w4.device_status() == 0


class Head:
    """A seeded LM head on the grid, and its logits."""

    def __init__(self, m, n, k, group=64, symmetric=False, seed=0):
        g = np.random.RandomState(seed)
        self.m, self.n, self.k, self.group = m, n, k, group
        self.x = np.clip(np.round(g.standard_normal((m, k)) * 8), -32, 32) / 8.0
        q = g.randint(0, 16, (n, k))
        steps = g.randint(4, 41, (n, k // group))
        bias = -8 * steps if symmetric else -8 * steps + g.randint(-2, 3, steps.shape)
        w = (steps[:, :, None] * q.reshape(n, -1, group) + bias[:, :, None]).reshape(n, k) * 2.0**-11
        self.logits = (self.x @ w.T).astype(np.float32)     # exact
        packed = np.zeros((n, k // 8), np.uint32)
        for i in range(8):
            packed |= q[:, i::8].astype(np.uint32) << np.uint32(4 * i)
        self.dev = (to_dev(self.x.astype(np.float16)), to_dev(packed), to_dev((steps * 2.0**-11).astype(np.float16)),
                    None if symmetric else to_dev((bias * 2.0**-11).astype(np.float16)))

    def pick(self, w4, top, rules=None, **kw):
        idx, val = w4.lm_head_argmax_topk(*self.dev, k=top, group=self.group, rules=rules, **kw)
        return idx.cpu().numpy(), val.cpu().numpy()


def ruled(logits, counts=None, slots=None, rep=None, pres=None, freq=None, biases=None, allowed=None):
    """The logits after the rules, in fp32 steps; masked ones are None (a bool mask beside them)."""
    z = logits.copy()
    m, n = z.shape
    if counts is not None:
        for r in range(m):
            if not 0 <= slots[r] < len(counts):
                continue
            c = counts[slots[r]]
            seen, t = c != 0, (c & 0x7FFF).astype(np.float32)
            p = np.float32(1 if rep is None else rep[r])
            with np.errstate(divide="ignore", invalid="ignore"):
                z[r] = np.where(seen, np.where(z[r] > 0, z[r] / p, z[r] * p), z[r])
            f, q = np.float32(0 if freq is None else freq[r]), np.float32(0 if pres is None else pres[r])
            z[r] = np.where(t > 0, (z[r] - f * t) - q, z[r])
    if biases is not None:
        offsets, tokens, values = biases
        for r in range(m):
            lo, hi = offsets[r], offsets[r + 1]
            if not 0 <= lo <= hi <= len(tokens):
                continue
            for t in np.unique(tokens[lo:hi]):
                if 0 <= t < n:
                    z[r, t] = z[r, t] + np.float32(np.sum(values[lo:hi][tokens[lo:hi] == t].astype(np.float32)))
    left = np.ones((m, n), bool) if allowed is None else allowed
    return z, left


def best(z, left, top):
    idx, val = np.full((len(z), top), -1, np.int32), np.full((len(z), top), -np.inf, np.float32)
    for r in range(len(z)):
        at = np.flatnonzero(left[r])
        at = at[np.lexsort((at, -z[r, at].astype(np.float64)))][:top]
        idx[r, :len(at)], val[r, :len(at)] = at, z[r, at]
    return idx, val


def bits(allowed):
    m, n = allowed.shape
    wide = np.zeros((m, (n + 31) // 32 * 32), bool)
    wide[:, :n] = allowed
    # (bits past the vocabulary are ones in some rows: they do not matter)
    wide[::2, n:] = True
    return np.packbits(wide.reshape(m, -1, 32), axis=2, bitorder="little").view(np.uint32).reshape(m, -1).astype(np.uint32)


def check(w4, head, top, rule, rules):
    idx, val = head.pick(w4, top, rules)
    want_idx, want_val = best(*ruled(head.logits, **rule), top)
    assert np.array_equal(idx, want_idx)
    assert np.array_equal(val.view(np.uint32), (want_val + np.float32(0)).view(np.uint32))


def counts_on(w4, counts, layout):
    import torch
    slots, n = counts.shape
    if layout == "new":
        t = w4.TokenCounts.new(slots, n)
        t.counts.copy_(to_dev(counts.view(np.int16)))
        return t
    pad = 3 if layout == "odd" else 8
    wide = torch.full((slots, n + pad), 77, dtype=torch.int16, device="cuda")
    part = wide[:, 1:n + 1] if layout == "odd" else wide[:, :n]
    part.copy_(to_dev(counts.view(np.int16)))
    return w4.TokenCounts(part)


def random_rule(g, m, n, slots, density, with_bias=True, with_mask=True):
    counts = np.where(g.random_sample((slots, n)) < density, g.randint(1, 1 << 16, (slots, n)), 0).astype(np.uint16)
    rule = dict(counts=counts, slots=g.permutation(slots)[:m].astype(np.int32),
                rep=g.choice([1.0, 1.1, 1.3, 0.7], m).astype(np.float32),
                pres=g.choice([0.0, 0.5, 1.7], m).astype(np.float32),
                freq=g.choice([0.0, 0.001, 0.3], m).astype(np.float32))
    if with_bias:
        lens = g.randint(0, min(n, 300) + 1, m)
        offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        tokens = np.concatenate([g.permutation(n)[:c] for c in lens] or [[]]).astype(np.int32)
        rule["biases"] = (offsets, tokens, (g.randint(-40, 41, len(tokens)) / 4).astype(np.float32))
    if with_mask:
        share = g.choice([1.0, 0.5, 0.02], (m, 1))
        rule["allowed"] = g.random_sample((m, n)) < share
    return rule


def rules_of(w4, rule, layout="new"):
    kw = {}
    if "counts" in rule:
        kw["counts"] = counts_on(w4, rule["counts"], layout)
        kw["slots"] = to_dev(rule["slots"])
    for name, key in (("repetition", "rep"), ("presence", "pres"), ("frequency", "freq")):
        if key in rule:
            kw[name] = to_dev(rule[key])
    if "biases" in rule:
        kw["biases"] = tuple(to_dev(a) for a in rule["biases"])
    if "allowed" in rule:
        kw["allowed"] = to_dev(bits(rule["allowed"]).view(np.int32))
    return w4.LogitRules(**kw)


@pytest.mark.parametrize("m", [1, 2, 7, 9, 16])
@pytest.mark.parametrize("n,k,top", [(1, 64, 1), (5, 64, 5), (33, 128, 7), (1000, 896, 5), (5003, 256, 50), (5003, 256, 64),
                                     (20000, 192, 1)])
@pytest.mark.parametrize("layout", ["new", "odd", "even"])
def test_rules(w4, m, n, k, top, layout):
    head = Head(m, n, k, seed=m + n)
    g = np.random.RandomState(n + top)
    rule = random_rule(g, m, n, m + 2, 0.3)
    check(w4, head, top, rule, rules_of(w4, rule, layout))


@pytest.mark.parametrize("group,symmetric", [(64, False), (128, True), (32, False), (128, False)])
def test_rules_formats_and_full_vocabulary(w4, group, symmetric):
    for m, top in ((1, 1), (3, 50), (16, 20)):
        head = Head(m, 32008, 256, group, symmetric, seed=m)
        rule = random_rule(np.random.RandomState(m), m, 32008, m + 1, 0.05)
        check(w4, head, top, rule, rules_of(w4, rule))


@pytest.mark.parametrize("k", [64, 448, 960, 1024, 1088])
@pytest.mark.parametrize("m", [1, 2, 8, 9, 16])
def test_rules_of_many_narrow_tiles(w4, m, k):
    """Several tiles of four boxes and fewer a block, and of five, the last one ragged; with and without rules."""
    n = 16 * 304 * 2 + 1003
    head = Head(m, n, k, seed=k)
    rule = random_rule(np.random.RandomState(k), m, n, m + 1, 0.1)
    for top in (1, 30):
        check(w4, head, top, {}, None)
        check(w4, head, top, rule, rules_of(w4, rule))


@pytest.mark.parametrize("m", [7, 16])
def test_rules_at_the_widest_rows(w4, m):
    """Up to the largest K that a selection takes, where little shared memory is left for the rules."""
    import torch
    n = 1000

    def taken(k):
        x = torch.zeros(m, k, dtype=torch.float16, device="cuda")
        scales = torch.zeros(n, k // 64, dtype=torch.float16, device="cuda")
        try:
            w4.lm_head_argmax_topk(x, torch.zeros(n, k // 8, dtype=torch.int32, device="cuda"), scales, scales, k=5)
        except w4.W4A16Error as e:
            assert e.status == 2
            return False
        return True
    lo, hi = 64, 32768 + 64
    while hi - lo > 64:
        k = (lo + hi) // 128 * 64
        lo, hi = (k, hi) if taken(k) else (lo, k)
    assert 1024 <= lo <= 32768
    for k in (lo, lo - 64, lo - 192):
        head = Head(m, n, k, seed=k)
        rule = random_rule(np.random.RandomState(k), m, n, m + 1, 0.3)
        check(w4, head, 9, rule, rules_of(w4, rule))


def test_rules_parts_alone(w4):
    head = Head(5, 3001, 128, seed=3)
    full = random_rule(np.random.RandomState(8), 5, 3001, 9, 0.4)
    for keep in (["counts", "slots", "rep"], ["counts", "slots", "pres"], ["counts", "slots", "freq"], ["counts", "slots"],
                 ["biases"], ["allowed"], ["biases", "allowed"], []):
        rule = {k: full[k] for k in keep}
        check(w4, head, 30, rule, rules_of(w4, rule))
    plain = head.pick(w4, 30)
    for a, b in zip(plain, head.pick(w4, 30, w4.LogitRules())):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("top", [1, 2, 50, 64])
def test_masks_that_leave_little_or_nothing(w4, top):
    m, n = 6, 9001
    head = Head(m, n, 128, seed=1)
    allowed = np.zeros((m, n), bool)
    allowed[1, n - 1] = True
    allowed[2, 0] = True
    allowed[3, :top - 1] = True
    allowed[4, 100:100 + top] = True
    allowed[5] = True
    check(w4, head, top, dict(allowed=allowed), rules_of(w4, dict(allowed=allowed)))
    assert w4.device_status() == 0


def test_infinite_and_equal_logits(w4):
    """Biases of -inf come last but can be selected, +inf first; equal logits go to the lowest index that is allowed,
    also where thousands are equal."""
    m, n = 3, 6000
    head = Head(m, n, 64, seed=2)
    head.dev[0].zero_()
    head.logits[:] = 0
    allowed = np.ones((m, n), bool)
    allowed[0, :50] = False
    allowed[1, ::2] = False
    rule = dict(allowed=allowed)
    for top in (1, 50):
        check(w4, head, top, rule, rules_of(w4, rule))
    head = Head(m, 40, 64, seed=4)
    tokens = np.concatenate([np.arange(40), [3], [7, 9, 39]]).astype(np.int32)
    values = np.concatenate([np.full(40, -np.inf), [np.inf], [np.inf, -np.inf, np.inf]]).astype(np.float32)
    rule = dict(biases=(np.array([0, 40, 41, 44], np.int32), tokens, values))
    check(w4, head, 40, rule, rules_of(w4, rule))


def test_biases_of_one_token_add_up(w4):
    """The same token many times in a list: inside one chunk of 32 entries and across chunks (values whose sums are exact)."""
    g = np.random.RandomState(5)
    m, n = 4, 700
    head = Head(m, n, 64, seed=5)
    lens = [0, 1, 33, 1000]
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = g.randint(-3, 40, offsets[-1]).astype(np.int32)      # negative ones are skipped
    values = (g.randint(-40, 41, offsets[-1]) / 8).astype(np.float32)
    rule = dict(biases=(offsets, tokens, values))
    check(w4, head, 40, rule, rules_of(w4, rule))
    assert w4.device_status() == 0


def added_in_order(logits, biases):
    """Every entry of a list added to its token's logit, one fp32 addition after the other."""
    z = logits.copy()
    offsets, tokens, values = biases
    for r in range(len(z)):
        for i in range(offsets[r], offsets[r + 1]):
            if tokens[i] >= 0:
                z[r, tokens[i]] = np.float32(z[r, tokens[i]] + values[i])
    return z


@pytest.mark.parametrize("lens", [(200, 0, 0), (33, 64, 7), (200, 300, 0), (1, 200, 1000)])
def test_biases_of_one_token_round_in_order(w4, lens):
    """Entries of one token whose sums are not exact and that cancel, in one chunk of 32 and across chunks, in lists of
    few entries a block and of many: bit for bit as in the definition, whatever the other rows' lists hold."""
    g = np.random.RandomState(sum(lens))
    m, n = 3, 48
    head = Head(m, n, 64, seed=11)
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = g.randint(-2, 12, offsets[-1]).astype(np.int32)
    tokens[::9] += 30
    values = (g.standard_normal(offsets[-1]) * 10.0 ** g.randint(-3, 8, offsets[-1])).astype(np.float32)
    values[2::6] = 1e8
    values[5::6] = -1e8
    biases = (offsets, tokens, values)
    want = best(added_in_order(head.logits, biases), np.ones((m, n), bool), n)
    idx, val = head.pick(w4, n, rules_of(w4, dict(biases=biases)))
    assert np.array_equal(val.view(np.uint32), (want[1] + np.float32(0)).view(np.uint32))
    assert np.array_equal(idx, want[0])


def test_bad_indexes_are_skipped_and_reported(w4):
    m, n = 4, 500
    head = Head(m, n, 64, seed=6)
    g = np.random.RandomState(6)
    counts = np.where(g.random_sample((3, n)) < 0.5, 5, 0).astype(np.uint16)
    rule = dict(counts=counts, slots=np.array([2, -1, 3, 2**31 - 1], np.int32), rep=np.full(m, 1.5, np.float32))
    check(w4, head, 20, rule, rules_of(w4, rule))
    assert w4.device_status() == 9 and w4.device_status() == 0
    rule["slots"] = np.array([2, -1, 0, -(2**31)], np.int32)     # negative ones are no mistake
    check(w4, head, 20, rule, rules_of(w4, rule))
    assert w4.device_status() == 0
    tokens, values = np.array([1, n, 2, 2**31 - 1], np.int32), np.full(4, 100, np.float32)
    for offsets, bad in (([0, 2, 4, 4, 4], True), ([0, 1, 5, 4, 4], True), ([-1, 1, 1, 1, 1], True), ([3, 2, 1, 1, 1], True)):
        rule = dict(biases=(np.array(offsets, np.int32), tokens, values))
        check(w4, head, 20, rule, rules_of(w4, rule))
        assert w4.device_status() == (9 if bad else 0) and w4.device_status() == 0


def test_captured_and_replayed_with_other_contents(w4):
    import torch
    m, n = 3, 4000
    head = Head(m, n, 128, seed=7)
    rule = random_rule(np.random.RandomState(1), m, n, 5, 0.3, with_bias=False)
    rules = rules_of(w4, rule)
    x, qw, s, b = head.dev
    idx, val = torch.zeros(m, 9, dtype=torch.int32, device="cuda"), torch.zeros(m, 9, device="cuda")
    ws = torch.empty(w4.lm_head_workspace_bytes(m, n, 9), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.lm_head_argmax_topk(x, qw, s, b, k=9, idx=idx, val=val, workspace=ws, rules=rules)
        w4.token_counts_add(rules.counts, rules.tensors[1], idx[:, 0].contiguous())
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want_idx, want_val = best(*ruled(head.logits, **rule), 9)
        assert np.array_equal(idx.cpu().numpy(), want_idx) and np.array_equal(val.cpu().numpy(), want_val)
        for r in range(m):
            c = rule["counts"][rule["slots"][r]]
            t = want_idx[r, 0]
            if t >= 0:
                c[t] = (c[t] & 0x8000) | min((c[t] & 0x7FFF) + 1, 0x7FFF)
        assert np.array_equal(rules.counts.counts.cpu().numpy().view(np.uint16), rule["counts"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = w4.lm_head_argmax_topk(x, qw, s, b, k=9, rules=rules)
    side.synchronize()
    want_idx, _ = best(*ruled(head.logits, **rule), 9)
    assert np.array_equal(got.cpu().numpy(), want_idx)


def test_outputs_of_a_call_on_another_stream(w4):
    """Memory that the current stream has freed but not finished with does not become another stream's output."""
    import torch
    head = Head(2, 700, 64, seed=3)
    rule = random_rule(np.random.RandomState(3), 2, 700, 3, 0.3)
    rules = rules_of(w4, rule)
    want = best(*ruled(head.logits, **rule), 4)
    x, qw, s, b = head.dev
    side = torch.cuda.Stream()
    for which in (rules, None):       # (loads the kernels, which waits for the GPU)
        head.pick(w4, 4, which)
    torch.cuda.synchronize()
    for which in (rules, None):
        torch.cuda._sleep(20000000)   # the current stream is busy for some ms
        late = [torch.full((2, 4), -9, dtype=dtype, device="cuda") for dtype in (torch.int32, torch.float32)]
        late.append(torch.full((w4.lm_head_workspace_bytes(2, 700, 4),), 255, dtype=torch.uint8, device="cuda"))
        del late                      # (its fills are still to come)
        idx, val = w4.lm_head_argmax_topk(x, qw, s, b, k=4, stream=side, rules=which)
        torch.cuda.synchronize()
        expect = want if which is not None else best(head.logits, np.ones((2, 700), bool), 4)
        assert np.array_equal(idx.cpu().numpy(), expect[0]) and np.array_equal(val.cpu().numpy(), expect[1])


# ------------------------------------------------------------ token counts

def counted(counts, n, slots, tokens, offsets, prompt, reset):
    c = counts.copy()
    batch = len(slots)
    for b in range(batch):
        if not 0 <= slots[b] < len(c):
            continue
        if reset:
            c[slots[b], :n] = 0
        lo, hi = (b, b + 1) if offsets is None else (int(offsets[b]), int(offsets[b + 1]))
        if not 0 <= lo <= hi <= len(tokens):
            continue
        for t in tokens[lo:hi]:
            if 0 <= t < n:
                v = int(c[slots[b], t])
                c[slots[b], t] = v | 0x8000 if prompt else (v & 0x8000) | min((v & 0x7FFF) + 1, 0x7FFF)
    return c


@pytest.mark.parametrize("n", [1, 7, 1000, 8192, 8193, 40003])
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("reset", [False, True])
def test_token_counts(w4, n, prompt, reset):
    import torch
    g = np.random.RandomState(n)
    for layout in ("new", "odd", "even"):
        slots_n = 6
        start = g.randint(0, 1 << 16, (slots_n, n)).astype(np.uint16)
        start[:, ::3] = 0
        start[:, ::5] = 0x7FFE
        t = counts_on(w4, start, layout)
        base = t.counts._base if t.counts._base is not None else t.counts
        before = base.clone()
        lens = [0, 1, 40, 3000, 17]
        offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        tokens = np.minimum((n ** g.random_sample(offsets[-1])).astype(np.int64) - 1, n - 1).astype(np.int32)
        tokens[::11] = -1
        slots = np.array([4, 0, 5, 1, -2], np.int32)
        w4.token_counts_add(t, to_dev(slots), to_dev(tokens), to_dev(offsets), prompt=prompt, reset=reset)
        want = counted(start, n, slots, tokens, offsets, prompt, reset)
        assert np.array_equal(t.counts.cpu().numpy().view(np.uint16), want)
        part = before.as_strided(t.counts.shape, t.counts.stride(), t.counts.storage_offset())
        part.copy_(t.counts)
        assert torch.equal(before, base)      # nothing beside the rows
    assert w4.device_status() == 0


def test_token_counts_of_a_step(w4):
    """One token a sequence; none (-1), the same slot twice, and counts at their end."""
    n = 300
    start = np.zeros((4, n), np.uint16)
    start[1, 7], start[2, 7] = 0x7FFF, 0xFFFF
    t = counts_on(w4, start, "new")
    slots, tokens = np.array([0, 1, 2, 3, 3, -1, 0], np.int32), np.array([-1, 7, 7, 9, 9, 5, 299], np.int32)
    w4.token_counts_add(t, to_dev(slots), to_dev(tokens))
    assert np.array_equal(t.counts.cpu().numpy().view(np.uint16), counted(start, n, slots, tokens, None, False, False))
    big = np.full(70000, 9, np.int32)
    offsets = np.array([0, 100, 70000], np.int32)
    t = counts_on(w4, start, "odd")
    w4.token_counts_add(t, to_dev(np.array([0, 3], np.int32)), to_dev(big), to_dev(offsets))
    got = t.counts.cpu().numpy().view(np.uint16)
    assert got[0, 9] == 100 and got[3, 9] == 0x7FFF and got.sum() == 100 + 0x7FFF + 0x7FFF + 0xFFFF
    w4.token_counts_add(t, to_dev(np.array([0, 3], np.int32)), to_dev(big), to_dev(offsets), reset=True)
    got = t.counts.cpu().numpy().view(np.uint16)
    assert got[0, 9] == 100 and got[3, 9] == 0x7FFF and got[0].sum() == 100
    assert w4.device_status() == 0


def test_token_counts_of_nothing(w4):
    """A step in which no request begins, and one whose requests bring no tokens."""
    import torch
    t = counts_on(w4, np.full((3, 50), 7, np.uint16), "new")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for prompt in (False, True):
        for reset in (False, True):
            w4.token_counts_add(t, none, none, prompt=prompt, reset=reset)
            w4.token_counts_add(t, none, none, offsets=zero, prompt=prompt, reset=reset)
            w4.token_counts_add(t, zero, none, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"), prompt=prompt)
    assert bool((t.counts == 7).all())
    w4.token_counts_add(t, zero + 2, none, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"), reset=True)
    assert bool((t.counts[:2] == 7).all()) and bool((t.counts[2] == 0).all())


def test_token_counts_bad_indexes(w4):
    n = 64
    start = np.zeros((3, n), np.uint16)
    ones = np.arange(8, dtype=np.int32)
    for slots, tokens, offsets in (([0, 3], ones, [0, 4, 8]), ([0, 1], np.where(ones == 2, n, ones), [0, 4, 8]),
                                   ([0, 1], ones, [0, 9, 8]), ([0, 1], ones, [0, 4, 9]), ([0, 1], ones, [-1, 4, 8]),
                                   ([0, 2**31 - 1], ones, [0, 4, 8])):
        for reset in (False, True):
            t = counts_on(w4, start, "new")
            slots, offsets = np.array(slots, np.int32), np.array(offsets, np.int32)
            w4.token_counts_add(t, to_dev(slots), to_dev(tokens), to_dev(offsets), reset=reset)
            got = t.counts.cpu().numpy().view(np.uint16)
            assert np.array_equal(got, counted(start, n, slots, tokens, offsets, False, reset)), (slots, offsets)
            assert w4.device_status() == 9 and w4.device_status() == 0


@pytest.mark.parametrize("slots,offsets", [([0, 1, 2], [0, 5, 3, 8]), ([0, 1, 2], [0, 8, 2, 8]), ([0, 9, 2], [0, 4, 4, 8]),
                                           ([0, 1, 9], [0, 4, 8, 8]), ([-1, 0, -1], [0, 3, 8, 6]), ([0, 2, -1], [0, 4, 8, 9])])
@pytest.mark.parametrize("reset", [False, True])
def test_token_counts_bad_sequences_without_tokens_of_their_own(w4, slots, offsets, reset):
    """Offsets out of order and slots past the last are reported, whether or not a token falls into their sequence; rows
    that no sequence names stay."""
    t = counts_on(w4, np.full((4, 40), 5, np.uint16), "new")
    w4.token_counts_add(t, to_dev(np.array(slots, np.int32)), to_dev(np.arange(8, dtype=np.int32)),
                        to_dev(np.array(offsets, np.int32)), reset=reset)
    assert w4.device_status() == 9 and w4.device_status() == 0
    got = t.counts.cpu().numpy()
    assert all((got[r] == 5).all() for r in range(4) if r not in slots)


def test_reset_of_one_slot_twice(w4):
    """The last of the sequences with one slot takes it, whole, whatever the others count; it is reported."""
    g = np.random.RandomState(5)
    n, batch = 20011, 301
    where = g.randint(0, 40, batch).astype(np.int32)
    where[-1] = where[0]
    lens = g.randint(0, 60, batch)
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens = g.randint(0, n, offsets[-1]).astype(np.int32)
    want = np.full((40, n), 3, np.int64)
    for b in range(batch):
        want[where[b]] = np.bincount(tokens[offsets[b]:offsets[b + 1]], minlength=n)
    for _ in range(3):
        table = to_dev(np.full((40, n), 3, np.int16))
        w4.token_counts_add(w4.TokenCounts(table), to_dev(where), to_dev(tokens), to_dev(offsets), reset=True)
        assert np.array_equal(table.cpu().numpy().astype(np.int64), want)
        assert w4.device_status() == 9 and w4.device_status() == 0


def test_wrong_rules_are_refused(w4):
    import torch
    head = Head(2, 100, 64, seed=9)
    counts = w4.TokenCounts.new(3, 100)
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    ones = torch.ones(2, device="cuda")
    with pytest.raises(TypeError):
        w4.TokenCounts(torch.zeros(3, 100, device="cuda"))
    with pytest.raises(ValueError):
        w4.TokenCounts(torch.zeros(3, 100, dtype=torch.int16))
    with pytest.raises(ValueError):
        w4.TokenCounts(torch.zeros(3, 100, dtype=torch.int16, device="cuda").T)
    with pytest.raises(ValueError):
        w4.LogitRules(counts)
    with pytest.raises(ValueError):
        w4.LogitRules(repetition=ones)
    with pytest.raises(ValueError):
        w4.LogitRules(counts, slots, repetition=ones[:1])
    with pytest.raises(TypeError):
        w4.LogitRules(counts, slots.long())
    with pytest.raises(ValueError):
        head.pick(w4, 5, w4.LogitRules(w4.TokenCounts.new(3, 99), slots))
    with pytest.raises(ValueError):
        head.pick(w4, 5, w4.LogitRules(counts, slots[:1]))
    with pytest.raises(ValueError):
        head.pick(w4, 5, w4.LogitRules(allowed=torch.zeros(2, 3, dtype=torch.int32, device="cuda")))
    with pytest.raises(ValueError):
        w4.LogitRules(biases=(torch.zeros(3, dtype=torch.int32, device="cuda"), slots, ones[:1]))
    with pytest.raises(ValueError):
        w4.token_counts_add(counts, slots, slots, offsets=slots)
    with pytest.raises(ValueError):
        w4.token_counts_add(counts, slots, slots[:1])
    with pytest.raises(TypeError):
        w4.token_counts_add(counts, slots, slots.long())
    empty = (torch.zeros(3, dtype=torch.int32, device="cuda"), slots[:0], ones[:0])
    head.pick(w4, 5, w4.LogitRules(biases=empty))
    assert w4.device_status() == 0
