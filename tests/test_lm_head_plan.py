"""What lm_head_argmax_topk would launch, from the planning code on the host: the ring of weights, and the shapes that
are taken."""
import ctypes

import pytest

from test_abi import lib  # noqa: F401  (the library fixture)

SMEM, SMS = 227 * 1024, 152


class Plan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int32) for name in ("blocks", "stages", "teams", "stage_bytes", "smem")]


@pytest.fixture(scope="module")
def plan(lib):  # noqa: F811
    f = lib.w4a16_testing_lm_head_plan
    f.argtypes = [ctypes.c_int] * 6 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]

    def of(m, n, k, group=64, symmetric=False, top=1, rules=None):
        p = Plan()
        status = f(m, n, k, group, int(symmetric), top, rules, SMS, ctypes.byref(p))
        return p if status == 0 else None
    return of


@pytest.mark.parametrize("m,n,k,stages", [(16, 151936, 2560, 3), (12, 151936, 4096, 3), (9, 151936, 6144, 3),
                                          (16, 32000, 4096, 3), (16, 151936, 2048, 4)])
def test_teams_leave_no_stage_of_the_ring_unused(plan, m, n, k, stages):
    """A ring of three stages is one team's."""
    p = plan(m, n, k)
    assert p.stages == stages and p.smem <= SMEM


def test_a_stage_belongs_to_one_team(plan):
    """Waits go by the parity of a phase, so a team must have seen the phase before in the same slot: the stages are a
    multiple of the teams; and where a tile has several chunks no team has to do with one."""
    most = set()
    for m in range(1, 17):
        for n in (1000, 50257, 151936, 262144, 340480, 384256):
            for k in (64, 512, 896, 1024, 2048, 2560, 4096, 5120, 6144):
                p = plan(m, n, k)
                if p:
                    assert p.stages % p.teams == 0 and p.stages >= (2 * p.teams if k > 2048 else p.teams), (m, n, k)
                    most.add((p.teams, min(p.stages, 5)))
    assert {(1, 2), (1, 3), (2, 4), (4, 5)} <= most


def aligned(n, to=16):
    return (n + to - 1) // to * to


def least_smem(m, n, k, group, symmetric, top):
    """What a block cannot do without: two stages of weights, its rows' activations and their sums, a tile's sums by
    warps (two tiles in turn, or all of them where these are few), and the logits."""
    blocks = min(-(-n // 16), min(SMS * (2 if m <= 8 else 1), 16384 // top))
    tiles, groups = -(-(-(-n // 16)) // blocks), k // 64
    stage = aligned(min(32, groups + 3) // 4 * 2048 + (32 if symmetric else 64) * (k // group), 1024)
    size = 2 * stage + aligned(groups * m * 128)
    size = aligned(size + groups * m * 4 * (2 if group == 32 else 1))
    size = aligned(size + min(2 * 8 * 16 * m * 4, tiles * 8 * 16 * m * 4))
    size = aligned(size + tiles * 16 * m * 4)
    return size + 16 * 2 + 16 + 1024


WIDE = [(7, 3648, 151936, 64, False), (11, 5760, 151936, 64, False), (14, 2816, 262144, 64, False),
        (6, 4992, 128256, 128, True), (16, 1024, 350000, 64, False), (16, 896, 396416, 64, False), (9, 1024, 778240, 64, False)]


@pytest.mark.parametrize("m,k,n,group,symmetric", WIDE)
def test_wide_selections_are_taken(plan, m, k, n, group, symmetric):
    p = plan(m, n, k, group, symmetric)
    assert p and p.smem <= SMEM // (2 if m <= 8 else 1)


@pytest.mark.parametrize("group,symmetric", [(64, False), (128, True), (32, False), (128, False), (32, True)])
def test_every_selection_that_fits_is_taken(plan, group, symmetric):
    taken = 0
    for n in (1000, 32000, 50257, 128256, 151936, 200064, 262144, 384256, 500009, 900000, 2000000):
        for m in range(1, 17):
            for top in (1, 5, 50, 64):
                if n * top > 1 << 24:
                    continue
                for k in (*range(128, 2049, 128), *range(2176, 17000, 256 if group > 64 else 192)):
                    fits = least_smem(m, n, k, group, symmetric, top) <= SMEM // (2 if m <= 8 else 1)
                    assert (plan(m, n, k, group, symmetric, top) is not None) == fits, (m, n, k, top)
                    taken += fits
    assert taken > 10000


class Rules(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("counts_stride", ctypes.c_int64), ("slot", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_offsets", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64), ("slots", ctypes.c_int32),
                ("bias_entries", ctypes.c_int32)]


RULED = [(16, 131072, 3584, 64, False), (6, 32000, 4032, 64, False), (4, 128256, 6912, 64, False), (3, 151936, 6976, 32, False),
         (2, 200064, 8960, 32, False), (16, 384256, 1024, 64, False)]


@pytest.mark.parametrize("group,symmetric", [(64, False), (128, True), (32, False)])
def test_rules_take_what_is_taken_without(plan, group, symmetric):
    there = ctypes.c_void_p(16)       # (only looked at as a pointer)
    mask = Rules(allowed=there, allowed_stride=1 << 20)
    every = Rules(there, 1 << 24, there, there, there, there, there, there, there, there, 1 << 20, 8, 999)
    shapes = [(m, n, k) for n in (1000, 32000, 128256, 151936, 200064, 262144) for m in range(1, 17)
              for k in range(128, 17000, 128)]
    shapes += [(m, n, k) for m, n, k, g, s in RULED if (g, s) == (group, symmetric)]
    taken = 0
    for m, n, k in shapes:
        plain = plan(m, n, k, group, symmetric, 5)
        for rules in (mask, every):
            p = plan(m, n, k, group, symmetric, 5, ctypes.byref(rules))
            assert (p is None) == (plain is None), (m, n, k)
        taken += plain is not None
    assert taken > 2000
