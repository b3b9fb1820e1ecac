"""Host-only: which single-position products make their codes themselves, told by the scratch
that they need, and that a call is held to it.  No test here launches a kernel."""
import pytest

import conv2d_backward_amd as gi
from test_gated_boundary import call
from test_sequence_boundary import lib  # noqa: F401  (a fixture)

F32, BF16, F16 = range(3)


def scratch(dtype, B, D, E):
    return gi.load_library().project_int8_step_workspace_for(dtype, B, D, E)


def test_many_numbers_for_a_thread_have_their_codes_made_before(lib):  # noqa: F811
    for B, D in ((5, 5400), (5, 6500), (9, 2700), (9, 3640), (2, 16385), (3, 10923), (17, 128), (1, 32769)):
        for dtype in (F32, BF16, F16):
            assert scratch(dtype, B, D, 4096) > 0, (B, D)
    for B, D in ((1, 32768), (2, 16384), (4, 4096), (7, 2048), (9, 1024), (16, 1024)):
        for dtype in (F32, BF16, F16):
            assert scratch(dtype, B, D, 4096) == 0, (B, D)
    for B, D in ((8, 4096), (16, 2048), (9, 2048), (3, 10900), (4, 8192), (5, 2049)):   # float32 has half the room
        assert scratch(F32, B, D, 4096) > 0 == scratch(BF16, B, D, 4096) == scratch(F16, B, D, 4096), (B, D)


def test_wide_outputs_have_their_codes_made_before(lib):  # noqa: F811
    for dtype in (F32, BF16, F16):
        assert scratch(dtype, 1, 2048, 16384) == 0 < scratch(dtype, 1, 2048, 16385)
        assert scratch(dtype, 5, 512, 16384) == 0 < scratch(dtype, 5, 512, 16385)
        assert scratch(dtype, 16, 128, 131072) > 0


def test_scratch_for_any_type_is_the_larger(lib):  # noqa: F811
    f = gi.load_library().project_int8_step_workspace
    for B, D, E in ((8, 4096, 4096), (1, 2048, 131072), (3, 500, 70), (300, 200, 10), (16, 2048, 16384)):
        assert f(B, D, E) == max(scratch(t, B, D, E) for t in (F32, BF16, F16))
    assert f(2, 70000, 10) == scratch(BF16, 2, 70000, 10) == scratch(3, 2, 4, 10) == scratch(F32, 0, 4, 10) == -1


@pytest.mark.parametrize("dtype", (F32, BF16, F16))
@pytest.mark.parametrize("B,D,E", [(9, 3640, 4096), (1, 2048, 16385), (16, 2049, 16)])
def test_refuses_too_little(lib, B, D, E, dtype):  # noqa: F811
    """(Only refusals: a call with enough would follow the fake pointers.)"""
    K = -(-D // 128) * 128
    needed = scratch(dtype, B, D, E)
    assert needed == B * (K + 4)
    sizes = {"B": B, "D": D, "E": E, "K": K, "dtype": dtype, "y.batch": E, "y.channel": 1}
    assert call("project_int8_step", workspace=0, **sizes) == gi.EINVAL
    assert call("project_int8_step", workspace_bytes=needed - 1, **sizes) == gi.EINVAL
