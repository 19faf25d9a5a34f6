"""The rotation tables of stretched contexts, from how often a pair turns (CPU)."""
import math
import os

import numpy as np
import pytest

from conftest import ROOT


@pytest.fixture(scope="module")
def w4():
    pytest.importorskip("torch")
    if not os.path.exists(os.path.join(ROOT, "int4_weight_only_affine_gb300", "libw4a16.so")):
        import __graft_entry__
        __graft_entry__.build()
    import int4_weight_only_affine_gb300 as w4
    return w4


def angles(w4, *args, **kw):
    turns, factor = w4.rope_turns(*args, device="cpu", **kw)
    return turns.numpy().view(np.uint64).astype(np.float64) * 2.0**-64 * 2 * np.pi, factor


@pytest.mark.parametrize("rot,base,length", [(128, 1e4, 131072), (128, 1e4, 70000), (128, 1e4, 62000), (64, 1e4, 131072),
                                             (64, 500.0, 8192), (32, 1e4, 4096), (128, 1e4, 4096), (128, 1e6, 32768),
                                             (16, 100.0, 100000)])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (16.0, 2.0)])
def test_yarn_from_turns_per_pair(w4, rot, base, length, fast, slow):
    """Pair i (of as many as the progression has, not only the head's) turns length * base**(-2 i / rot) / 2 pi times over
    the original context.  The ramp runs from the last whole i that turns `fast` times or more to the first that turns
    `slow` times or fewer, within 0 .. rot - 1, whether or not the head has that pair."""
    turns = [length * base ** (-2.0 * i / rot) / (2 * math.pi) for i in range(rot)]
    lo = max([i for i in range(rot) if turns[i] >= fast], default=0)
    hi = min([i for i in range(rot) if turns[i] <= slow], default=rot - 1)
    stretch = 4.0
    got, factor = angles(w4, rot, base, "yarn", stretch, length, fast, slow)
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        share = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
        want = theta * (1 - share) + theta / stretch * share
        assert abs(got[i] - want) <= 1e-12 * want, (i, got[i] / theta, want / theta)
        if turns[i] >= fast:
            assert abs(got[i] - theta) <= 1e-12 * theta
        if turns[i] > slow and i > lo:   # turns more often than that: not stretched in full
            assert got[i] > theta / stretch * (1 + 1e-6)
    assert factor == 0.1 * math.log(stretch) + 1.0


def test_yarn_of_a_long_original_context(w4):
    """rot 128, base 10**4, 131072 positions: the ramp begins at pair 45 (33 turns) and would end at 70 (0.9 turns); the
    last pair, 63 (2.4 turns), is 18 / 25 of the way."""
    got, _ = angles(w4, 128, 1e4, "yarn", 4.0, 131072)
    last = 1e4 ** (-126 / 128)
    assert abs(got[63] - last * (1 - 0.75 * 18 / 25)) <= 1e-12 * last
