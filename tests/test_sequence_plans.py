"""Host-only: the plan queries, and that the cases of test_gpu_sequence_plans.py get the
plans they name and name every one there is."""
import os
import re

import pytest

import conv2d_backward_amd as gi
from test_gpu_sequence_plans import BACKWARD, FORWARD

CSRC = os.path.join(os.path.dirname(os.path.abspath(gi.__file__)), "csrc")


def backward_plan(sizes):
    """The plan without the number of segments, and whether rows are cut."""
    p = gi.state_scan_plan(*sizes, backward=True)
    segments = int(re.search(r" segments=(\d+)", p).group(1))
    return re.sub(r" segments=\d+", "", p), "cut" if segments > 1 else "whole"


@pytest.mark.parametrize("plan,sizes", FORWARD, ids=str)
def test_forward_cases_get_their_plan(plan, sizes):
    """And have more states than a stage, and more than one chunk."""
    assert gi.state_scan_plan(*sizes) == plan
    lanes, positions, staged = (int(re.search(r"%s=(\d+)" % k, plan).group(1)) for k in ("lanes", "positions", "staged"))
    assert sizes[3] > staged and sizes[2] > lanes * positions


@pytest.mark.parametrize("plan,rows,sizes", BACKWARD, ids=str)
def test_backward_cases_get_their_plan(plan, rows, sizes):
    assert backward_plan(sizes) == (plan, rows)
    assert sizes[3] > 16


def test_no_forward_deal_is_left_out():
    text = open(os.path.join(CSRC, "kernels_state_scan.hip")).read()
    table = re.search(r"kDeals\[\] = \{(.*?)\};", text, re.S).group(1)
    deals = {tuple(map(int, d)) for d in re.findall(r"\{(\d+), (\d+), (\d+), (\d+)\}", table)}
    named = {tuple(map(int, re.findall(r"=(\d+)", plan)[:4])) for plan, _ in FORWARD}
    assert named == deals and len(deals) == 10


def test_no_backward_plan_is_left_out():
    """Over a wide sweep of sizes no plan comes up that no case has."""
    named = {(plan, rows) for plan, rows, _ in BACKWARD}
    seen = {backward_plan((B, G * Dg, L, N, G))
            for B in (1, 2, 5, 16, 300) for G in (1, 2, 32) for Dg in (1, 7, 20, 33, 64, 500, 4000)
            for L in (1, 15, 100, 128, 129, 257, 777, 2048, 8192) for N in (1, 3, 16, 24, 64, 129, 192, 256)
            if B * G * Dg < 1 << 24 and B * G * N * (L + 256) <= 1 << 30}
    assert seen == named


def test_refusals():
    for sizes in ((0, 4, 5, 3, 1), (1, 4, 5, 3, 3), (1, 4, 5, 300, 1)):
        for backward in (False, True):
            with pytest.raises(gi.Conv2dGiError):
                gi.state_scan_plan(*sizes, backward=backward)
