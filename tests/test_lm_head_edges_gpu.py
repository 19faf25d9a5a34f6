"""lm_head_argmax_topk where its ring of weights is short: long rows, many tiles a block, the last shapes that are taken.

Weights and activations on coarse grids, made and multiplied on the device: every sum of products is exact in fp32 in
any order, so the selection is known exactly."""
import ctypes

import pytest

from _gpu import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    require_gpu()
    import int4_weight_only_affine_gb300 as w4
    yield w4
    assert w4.device_status() == 0


class Head:
    def __init__(self, m, n, k, group=64, symmetric=False, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.m, self.n, self.k, self.group = m, n, k, group
        x = (torch.randn(m, k, generator=g, device="cuda") * 8).round_().clamp_(-32, 32).div_(8)
        qw = torch.randint(-2**31, 2**31, (n, k // 8), generator=g, device="cuda", dtype=torch.int32)
        steps = torch.randint(4, 41, (n, k // group), generator=g, device="cuda").float()
        bias = -8 * steps
        if not symmetric:
            bias += torch.randint(-2, 3, steps.shape, generator=g, device="cuda")
        self.logits = torch.empty(m, n, device="cuda")
        shifts = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
        for at in range(0, n, 8192):
            rows = slice(at, min(at + 8192, n))
            q = ((qw[rows, :, None] >> shifts) & 15).reshape(-1, k // group, group).float()
            w = (q * steps[rows, :, None] + bias[rows, :, None]).reshape(-1, k) * 2.0**-11
            self.logits[:, rows] = x @ w.T
        self.dev = (x.half(), qw, (steps * 2.0**-11).half(), None if symmetric else (bias * 2.0**-11).half())

    def check(self, w4, top, logits=None, **kw):
        import torch
        idx, val = w4.lm_head_argmax_topk(*self.dev, k=top, group=self.group, **kw)
        want, at = torch.sort(self.logits if logits is None else logits, dim=1, descending=True, stable=True)
        assert torch.equal(val, want[:, :top]) and torch.equal(idx, at[:, :top].int())


@pytest.mark.parametrize("m", [9, 16])
@pytest.mark.parametrize("k", [2112, 4096, 4160])
@pytest.mark.parametrize("n", [16 * 152 + 5, 16 * 152 * 2, 16 * 152 * 3 + 11])
def test_two_teams_over_several_chunks(w4, m, k, n):
    """One, two and three or four tiles a block, for two teams, of two or three chunks of K each."""
    head = Head(m, n, k, seed=n + k)
    for top in (1, 20):
        head.check(w4, top)


@pytest.mark.parametrize("m,n,k", [(16, 151936, 2560), (9, 151936, 6144), (12, 32000, 5120), (9, 32000, 8192)])
def test_two_teams_with_two_or_three_stages(w4, m, n, k):
    head = Head(m, n, k, seed=m)
    for top in (1, 50):
        head.check(w4, top)


def last_taken(w4, m, k, group, symmetric, top, most):
    """The largest vocabulary that is taken, from the plan on the host (w4a16_testing_lm_head: five numbers)."""
    import torch
    f = w4.lib.w4a16_testing_lm_head_plan
    f.argtypes = [ctypes.c_int] * 6 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    out, sms = (ctypes.c_int32 * 5)(), torch.cuda.get_device_properties(0).multi_processor_count
    lo, hi = top, most
    while hi - lo > 1:
        n = (lo + hi) // 2
        lo, hi = (n, hi) if f(m, n, k, group, int(symmetric), top, None, sms, out) == 0 else (lo, n)
    return lo


@pytest.mark.parametrize("m,k,group,symmetric,top", [(1, 64, 64, False, 2), (3, 64, 64, False, 1), (8, 128, 64, False, 5),
                                                     (9, 256, 32, False, 3), (16, 1024, 64, False, 20), (16, 1024, 64, False, 1),
                                                     (12, 896, 128, True, 50), (7, 3648, 64, False, 9), (16, 2816, 64, False, 1)])
def test_the_widest_vocabulary(w4, m, k, group, symmetric, top):
    n = last_taken(w4, m, k, group, symmetric, top, (1 << 24) // top)
    assert n > 100000
    head = Head(m, n, k, group, symmetric, seed=m)
    head.check(w4, top)


@pytest.mark.parametrize("m,n,k,group,symmetric", [(7, 151936, 3648, 64, False), (11, 151936, 5760, 64, False),
                                                   (14, 262144, 2816, 64, False), (6, 128256, 4992, 128, True),
                                                   (16, 350000, 1024, 64, False)])
def test_wide_vocabularies(w4, m, n, k, group, symmetric):
    head = Head(m, n, k, group, symmetric, seed=m)
    for top in (1, 30):
        head.check(w4, top)


def ruled(head, seed, mask_only):
    """Rules for a head's rows, and its logits after them (fp32 steps; masked ones are -infinity)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n, z = head.m, head.n, head.logits.clone()
    kw = {}
    if not mask_only:
        counts = torch.randint(-2**15, 2**15, (m + 2, n), generator=g, device="cuda", dtype=torch.int16)
        counts[torch.rand(m + 2, n, generator=g, device="cuda") < 0.8] = 0
        kw["counts"], kw["slots"] = counts, torch.randperm(m + 2, generator=g, device="cuda")[:m].int()
        kw["repetition"] = 1 + 0.05 * torch.randint(0, 8, (m,), generator=g, device="cuda")
        kw["presence"] = 0.125 * torch.randint(0, 5, (m,), generator=g, device="cuda")
        kw["frequency"] = 0.001 * torch.randint(0, 5, (m,), generator=g, device="cuda")
        c = counts[kw["slots"].long()]
        t, rep = (c & 0x7FFF).float(), kw["repetition"][:, None]
        z = torch.where(c != 0, torch.where(z > 0, z / rep, z * rep), z)
        z = torch.where(t > 0, (z - kw["frequency"][:, None] * t) - kw["presence"][:, None], z)
        tokens = torch.stack([torch.randperm(n, generator=g, device="cuda")[:300] for _ in range(m)])
        values = 0.25 * torch.randint(-40, 41, tokens.shape, generator=g, device="cuda")
        z.scatter_add_(1, tokens, values)
        offsets = (300 * torch.arange(m + 1, device="cuda")).int()
        kw["biases"] = (offsets, tokens.int().reshape(-1), values.reshape(-1))
    allowed = torch.rand(m, (n + 31) // 32 * 32, generator=g, device="cuda") < 0.5
    bits = (allowed.view(m, -1, 32).long() << torch.arange(32, device="cuda")).sum(-1)
    kw["allowed"] = bits.to(torch.int32)
    return kw, z.masked_fill(~allowed[:, :n], float("-inf"))


@pytest.mark.parametrize("m,n,k,group", [(16, 131072, 3584, 64), (6, 32000, 4032, 64), (4, 128256, 6912, 64), (3, 151936, 6976, 32),
                                         (2, 200064, 8960, 32), (16, 384256, 1024, 64), (9, 890112, 256, 32)])
def test_rules_on_the_widest_selections(w4, m, n, k, group):
    """Where the rules have no shared memory of their own."""
    head = Head(m, n, k, group, seed=k)
    for mask_only in (True, False):
        kw, z = ruled(head, m, mask_only)
        if not mask_only:
            kw["counts"] = w4.TokenCounts(kw["counts"])
        for top in (1, 17):
            head.check(w4, top, z, rules=w4.LogitRules(**kw))
