"""Batches over a paged cache and their 64-bit oracle, for the attention tests
(not collected: no test_ prefix).

The oracle restates the definitions with numpy in binary64 and shares no code
with the library: rotation by complex multiplication with cos/sin of
position * theta, attention by a dense softmax per sequence and head."""
import math

import numpy as np

U16 = 2.0**-11   # binary16 unit roundoff
TINY16 = 2.0**-25  # half the smallest binary16 subnormal


def thetas(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def turns_of(theta):
    """int64 fractions of a turn, 2**64 to a turn."""
    return np.array([round(float(t) / (2 * math.pi) * 2.0**64) % 2**64 for t in theta], np.uint64).view(np.int64)


def rotate(x, positions, theta, factor=1.0, interleaved=False):
    """binary64 rotation of x [tokens][heads][dim]."""
    x = x.astype(np.float64)
    n = len(theta)
    even = np.arange(n) * 2 if interleaved else np.arange(n)
    odd = even + 1 if interleaved else even + n
    z = (x[..., even] + 1j * x[..., odd]) * factor * np.exp(1j * np.outer(positions, theta))[:, None, :]
    y = x.copy()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def rotate_tol(x, positions, theta, factor=1.0, interleaved=False):
    """Bound on |gpu - oracle|: one binary16 rounding of the result, and fp32 products with sines of an angle
    that is off by at most 2**-22 (the fraction of a turn in 24 bits times 2 pi, sincospif to 2 ulp)."""
    y = rotate(x, positions, theta, factor, interleaved)
    size = np.abs(x.astype(np.float64))
    n = len(theta)
    even = np.arange(n) * 2 if interleaved else np.arange(n)
    odd = even + 1 if interleaved else even + n
    pair = np.zeros_like(size)
    pair[..., even] = pair[..., odd] = (size[..., even] + size[..., odd]) * abs(factor)
    return U16 * np.abs(y) + 2.0**-20 * pair + TINY16


class Batch:
    """Sequences with q_lens new tokens and kv_lens cached ones, and a shuffled page table."""

    def __init__(self, q_lens, kv_lens, page, seed, spare=3, extra_rows=0):
        g = np.random.RandomState(seed)
        self.q_lens, self.kv_lens, self.page = np.array(q_lens), np.array(kv_lens), page
        need = -(-self.kv_lens // page)
        self.pages = int(need.sum()) + spare
        order = g.permutation(self.pages)
        self.table = np.full((len(q_lens), max(1, int(need.max()))), -7, np.int32)  # unused entries: no page
        n = 0
        for b, k in enumerate(need):
            self.table[b, :k] = order[n:n + k]
            n += k
        self.offsets = np.concatenate([[0], np.cumsum(self.q_lens)]).astype(np.int32)
        self.tokens = int(self.offsets[-1]) + extra_rows

    def positions(self, b):
        return np.arange(self.kv_lens[b] - self.q_lens[b], self.kv_lens[b])

    def slot(self, b, p):
        return self.table[b, p // self.page], p % self.page

    def used(self):
        """bool [pages][page]: slots that hold a position of a sequence."""
        m = np.zeros((self.pages, self.page), bool)
        for b in range(len(self.q_lens)):
            p = np.arange(self.kv_lens[b])
            m[self.slot(b, p)] = True
        return m


def seen(batch, b, causal, window):
    """bool [q_len][kv_len]: which positions each new token sees."""
    p = batch.positions(b)[:, None]
    j = np.arange(batch.kv_lens[b])[None]
    m = np.ones((len(p), j.shape[1]), bool)
    if causal:
        m &= j <= p
    if window:
        m &= j > p - window
    return m


def attention(q, kc, vc, batch, scale, causal=True, window=0):
    """(y, lse, tol_y, tol_lse) in binary64; rows outside every sequence are NaN.

    tol_y bounds |gpu - oracle| elementwise, with A = sum_j p_j |v_j| and n positions:
      probabilities rounded to binary16               U16 A + n TINY16 max|v|
      the result rounded to binary16                  U16 |y| + TINY16
      scores in fp32: (dim + 4) 2**-23 sum |q k| scale, as e: p is off by e relatively, and so is the sum: 2 e A
      exponentials (2 ulp of an argument up to 2**7)  2**-16 A covers both
      fp32 sums over n positions, 16 at a time        (n / 16 + 8) 2**-22 A
    """
    n_tok, hq, d = q.shape
    hkv = kc.shape[2]
    y = np.full((n_tok, hq, d), np.nan)
    lse = np.full((n_tok, hq), np.nan)
    ty, tl = y.copy(), lse.copy()
    for b in range(len(batch.q_lens)):
        rows = slice(batch.offsets[b], batch.offsets[b + 1])
        n = int(batch.kv_lens[b])
        m = seen(batch, b, causal, window)
        any_ = m.any(0)
        page, at = batch.slot(b, np.arange(n)) if n else (np.zeros(0, int),) * 2
        for h in range(hq):
            k = np.where(any_[:, None], kc[page, at, h * hkv // hq].astype(np.float64), 0.0)
            v = np.where(any_[:, None], vc[page, at, h * hkv // hq].astype(np.float64), 0.0)
            qh = q[rows, h].astype(np.float64)
            s = np.where(m, qh @ k.T * scale, -np.inf)
            e = (d + 4) * 2.0**-23 * scale * np.where(m, np.abs(qh) @ np.abs(k).T, 0.0).max(1, initial=0.0)
            top = s.max(1, initial=-np.inf)
            p = np.exp(s - np.where(np.isfinite(top), top, 0.0)[:, None])
            total = p.sum(1)
            p = p / np.where(total > 0, total, 1.0)[:, None]
            y[rows, h] = p @ v
            with np.errstate(divide="ignore"):
                lse[rows, h] = top + np.log(total)
            a = p @ np.abs(v)
            sums = (n / 16 + 8) * 2.0**-22
            ty[rows, h] = ((U16 + 2 * e[:, None] + 2.0**-16 + sums) * a + n * TINY16 * np.abs(v).max(initial=0.0)
                           + U16 * np.abs(y[rows, h]) + TINY16)
            with np.errstate(invalid="ignore"):
                tl[rows, h] = e + 2.0**-16 + sums + 2.0**-22 * np.abs(np.where(np.isfinite(lse[rows, h]), lse[rows, h], 0))
    return y, lse, ty, tl
