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
