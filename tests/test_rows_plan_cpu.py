"""How a group norm's work is cut and the workspace that it takes, asked of the
library for devices of a given size (no GPU)."""
import ctypes
import itertools
import random

import pytest

from row_wise_normalization_rmsnorm_gb300 import build as rn_build

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, F16, W32 = 0, 1, 2, 0x100


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("chunk", "cluster", "groups", "rows", "stages", "smem_bytes")] + \
        [("workspace_bytes", ctypes.c_int64)]


@pytest.fixture(scope="module")
def rn():
    rn_build.build()
    import row_wise_normalization_rmsnorm_gb300 as pkg
    return pkg


def plan(rn, B, S, C, G, dt, backward=0, kept=0, row=16, code=16, sms=152, most=16):
    p = Plan()
    assert rn.lib().groupnorm_plan_query(B, S, C, G, dt, backward, kept, row, code, sms, most, ctypes.byref(p)) == OK
    return p


def some_sizes(n):
    rng = random.Random(5)
    for _ in range(n):
        G = rng.choice([1, 2, 3, 4, 8, 9, 16, 32, 32, 32, 64])
        C = G * rng.choice([1, 3, 4, 6, 8, 10, 16, 20, 23, 30, 40, 64])
        yield rng.choice([1, 1, 2, 4, 8, 16, 300]), int(2 ** rng.uniform(0, 17)), C, G


# Sizes where a cluster holds the plain call's groups and none the keeping call's.
WINDOW = [(1, 16384, 320, 32, BF16), (4, 9216, 320, 32, BF16), (8, 5184, 320, 32, F16), (1, 9216, 640, 32, BF16), (4, 4096, 320, 32, F32),
          (16, 9216, 192, 32, BF16), (1, 1024, 736, 32, BF16)]


@pytest.mark.parametrize("B,S,C,G,dt", WINDOW)
def test_the_keeping_call_may_take_workspace_where_the_plain_one_takes_none(rn, B, S, C, G, dt):
    plain, keeping = plan(rn, B, S, C, G, dt), plan(rn, B, S, C, G, dt, kept=1)
    assert plain.cluster > 0 and plain.workspace_bytes == 0
    assert keeping.cluster == 0 and keeping.workspace_bytes > 0
    assert plan(rn, B, S, C, G, dt, row=0).workspace_bytes >= keeping.workspace_bytes


def test_the_workspace_that_is_asked_for_is_enough_for_every_call(rn):
    sizes = list(some_sizes(400)) + [w[:4] for w in WINDOW]
    for (B, S, C, G), dt, backward, sms in itertools.product(sizes, (F32, BF16), (0, 1), (148, 152)):
        most = plan(rn, B, S, C, G, dt, backward, row=0, sms=sms).workspace_bytes
        needs = [plan(rn, B, S, C, G, dt, backward, kept, row, code, sms).workspace_bytes
                 for kept in (0, 1) for row in (1, 2, 4, 8, 16) for code in (1, 2, 4, 8, 16)]
        assert max(needs) == most, (B, S, C, G, dt, backward)


def test_every_ring_has_a_stage_and_fits_an_sm(rn):
    """The widest rows with the most groups: a stage at least, in the shared memory that a CTA may have (227 KB, of
    which barriers and the mailbox take less than 1 KB)."""
    least = 9
    for C, G in [(C, G) for C in (8192, 8190, 8000, 7900, 5120, 4099, 2050, 1030) for G in (1, 2, 5, 10, C // 8, C // 4, C // 2, 4096)]:
        if C % G or G > 4096:
            continue
        for dt, backward, kept, row in itertools.product((F32, BF16), (0, 1), (0, 1), (1, 16)):
            p = plan(rn, 2, 30000, C, G, dt, backward, kept, row, row)
            assert p.smem_bytes <= 226 * 1024
            if p.cluster == 0:
                assert p.stages >= 1, (C, G, dt, backward, kept, row)
                least = min(least, p.stages)
    assert least == 1  # the fp32 gradient of 8192 channels in 4096 groups


def test_clusters_are_no_larger_than_the_device_holds(rn):
    """A device that holds no clusters of 16 (or 8 ...) is given smaller ones, or pieces."""
    seen = {most: set() for most in (1, 2, 4, 8, 16)}
    for B, S, C, G in some_sizes(300):
        for most, backward in itertools.product(seen, (0, 1)):
            p = plan(rn, B, S, C, G, BF16, backward, most=most)
            assert p.cluster <= most
            assert (p.cluster > 0) != (p.stages > 0)
            seen[most].add(p.cluster)
    assert all(max(seen[most]) == most and 0 in seen[most] for most in seen)


def test_plan_queries_refuse(rn):
    ask, p = rn.lib().groupnorm_plan_query, ctypes.byref(Plan())
    assert ask(1, 64, 64, 8, BF16, 0, 0, 16, 16, 152, 16, None) == INVALID
    for bad in ((-1, 64, 64, 8, BF16), (1, -1, 64, 8, BF16), (1, 64, 0, 8, BF16), (1, 64, 64, 7, BF16), (1, 64, 8200, 8, BF16),
                (1, 64, 64, 8, 5)):
        assert ask(*bad, 0, 0, 16, 16, 152, 16, p) == INVALID
    assert ask(1, 64, 64, 8, BF16, 0, 0, -1, 16, 152, 16, p) == INVALID
    assert ask(1, 64, 64, 8, BF16, 0, 0, 16, 16, -1, 16, p) == INVALID
    assert ask(1, 64, 64, 8, BF16, 0, 0, 16, 16, 152, 0, p) == INVALID
    assert ask(1, 64, 8192, 8192, BF16, 0, 0, 16, 16, 152, 16, p) == UNSUPPORTED
    for none in ((0, 64), (2, 0)):
        assert plan(rn, *none, 64, 8, BF16).workspace_bytes == 0


GIVE_UP = {"dy": None, "x": 4096, "mean": 4096, "rstd": 4096, "out": 4096, "B": 2, "S": 64, "C": 64, "G": 8, "dt": BF16, "sample": 0,
           "polls": 100, "stream": None}


@pytest.mark.parametrize("bad", [{"x": None}, {"out": None}, {"mean": None}, {"rstd": None}, {"x": 4097}, {"dy": 4097}, {"B": 0}, {"S": 0},
                                 {"G": 7}, {"dt": 5}, {"dt": BF16 | W32}, {"sample": 2}, {"sample": -1}, {"polls": 0}, {"C": 8192, "G": 8192}])
def test_the_check_of_a_wait_that_gives_up_refuses(rn, bad):
    assert rn.lib().groupnorm_give_up_check(*{**GIVE_UP, **bad}.values()) == INVALID
