"""Host-only: gated_scan's plan query, and that the GPU tests' cases come upon every plan there is,
forward and backward, and backward with all batch items in a work-group and with one."""
import ctypes

import pytest

import conv2d_backward_amd as gi

torch = pytest.importorskip("torch")
from test_sequence_boundary import lib  # noqa: E402,F401  (a fixture)

# Sizes of test_gpu_gated_scan.py by the plan that they are there for.
FORWARD = {
    "lanes=4 waves=1": (20, 7, 5), "lanes=16 waves=1": (3, 1400, 150), "lanes=64 waves=1": (1, 4100, 520),
    "lanes=64 waves=2": (1, 5, 513), "lanes=64 waves=4": (3, 4, 1030), "lanes=64 waves=8": (1, 3, 2049),
    "lanes=64 waves=16": (2, 1, 9001),
}


def gpu_module(name):
    return pytest.importorskip(name)


def whole(B, D, L):
    """Whether a backward work-group has all batch items: then the parameters' sums need no scratch."""
    scratch = gi.load_library().gated_scan_workspace
    scratch.restype = ctypes.c_int64
    return scratch(B, D, L) == 0


def sweep():
    return ((B, D, L) for B in (1, 2, 3, 5, 8, 16, 300) for D in (1, 7, 33, 256, 500, 1000, 2048, 4096, 16384)
            for L in (1, 31, 33, 128, 129, 500, 512, 513, 900, 1024, 1025, 2000, 2048, 3000, 4096, 8192, 20000, 100000))


def test_forward_cases_get_their_plan(lib):  # noqa: F811
    module = gpu_module("test_gpu_gated_scan")
    many = next(m for m in module.test_many_rows.pytestmark if m.name == "parametrize").args[1]
    cases = [tuple(c[:3]) for c in [*module.CASES, *many]]
    for plan, sizes in FORWARD.items():
        assert gi.gated_scan_plan(*sizes) == plan and sizes in cases


def test_backward_cases_get_their_plan(lib):  # noqa: F811
    for (plan, all_items), (B, D, L, _, _) in gpu_module("test_gpu_gated_shares").SHARES:
        assert (gi.gated_scan_plan(B, D, L, backward=True), whole(B, D, L)) == (plan, all_items), (B, D, L)


def test_no_plan_is_left_out(lib):  # noqa: F811
    """Over a wide sweep of sizes no plan comes up that no case has."""
    assert {gi.gated_scan_plan(*sizes) for sizes in sweep()} == set(FORWARD)
    seen = {(gi.gated_scan_plan(*sizes, backward=True), whole(*sizes)) for sizes in sweep()}
    assert seen == {plan for plan, _ in gpu_module("test_gpu_gated_shares").SHARES}
