"""What lm_head_argmax_topk would launch, from the planning code on the host: the ring of weights, and the shapes that
are taken."""
import ctypes

import pytest

from test_abi import lib  # noqa: F401  (the library fixture)

SMEM, SMS = 227 * 1024, 152


class Plan(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_int32), ("stages", ctypes.c_int32), ("stage_bytes", ctypes.c_int32), ("smem", ctypes.c_int32)]


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
    """Two teams of consumers share one ring: it need not have an even number of stages."""
    p = plan(m, n, k)
    assert p.stages == stages and p.smem <= SMEM
