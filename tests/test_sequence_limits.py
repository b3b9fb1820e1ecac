"""Host-side tests of the sequence operators' size limits: a call is refused for what its
own kernels cannot do.  As in test_sequence_boundary.py nothing is launched: a call that
is within the limits is refused for its output's strides, which are looked at later.
"""
import conv2d_backward_amd as gi
from test_sequence_boundary import call, lib, workspace  # noqa: F401  (lib: a fixture)

APART = {"y.channel": 0}   # EINVAL, after the sizes


def test_scan_calls_without_gradients_have_no_limit_of_the_gradients(lib):  # noqa: F811
    """B*G*N*(L+256) beyond 2^30, which bounds the sums of dB and dC."""
    assert call("state_scan_step", B=4200, D=64, G=8, N=128, lines=4200, **APART) == gi.EINVAL
    assert call("state_scan", B=64, D=64, G=8, N=128, L=16640, **APART) == gi.EINVAL
    assert call("state_scan_backward", B=64, D=64, G=8, N=128, L=1 << 18) == gi.EUNSUPPORTED
    assert workspace("state_scan_workspace", 64, 64, 1 << 18, 128, 8) == -1


def test_scan_forward_is_refused_beyond_its_own_grid(lib):  # noqa: F811
    """A work-group of 256 or 512 for each group of one channel: 2^32 work-items or more."""
    most = (1 << 24) - 1
    assert call("state_scan", B=1, D=most, G=most, N=256, L=1) == gi.EUNSUPPORTED
    assert call("state_scan", B=1, D=most, G=1, N=256, L=1, **APART) == gi.EINVAL


def test_scan_gradients_are_refused_for_the_whole_of_their_last_grid(lib):  # noqa: F811
    """The join of dB and dC has D*(N+2) work-items of its parameters behind them: counted
    too, or the first kernels of a call run and the last one's launch fails."""
    for sizes in (dict(B=1, D=(1 << 24) - 8, L=1, N=256, G=1),
                  dict(B=1, D=1 << 23, L=(1 << 22) - 512, N=256, G=1)):
        assert call("state_scan_backward", **sizes) == gi.EUNSUPPORTED
        assert workspace("state_scan_workspace", *(sizes[k] for k in "BDLNG")) == -1
    for sizes in (dict(B=1, D=(1 << 24) - 8, L=1, N=128, G=1),
                  dict(B=1, D=1 << 22, L=(1 << 22) - 512, N=256, G=1)):
        assert call("state_scan_backward", **{"dx.channel": 0}, **sizes) == gi.EINVAL
        assert workspace("state_scan_workspace", *(sizes[k] for k in "BDLNG")) > 0


def test_norm_is_refused_by_the_columns_its_work_groups_have(lib):  # noqa: F811
    """1024 work-items for 32 columns, for 16 of 1025 .. 2048 channels: 2^32 or more are refused."""
    for L, D, code in ((1 << 23, 1024, gi.EINVAL), (1 << 23, 1500, gi.EUNSUPPORTED), ((1 << 23) - 8, 1500, gi.EUNSUPPORTED),
                       ((1 << 23) - 16, 1500, gi.EINVAL), (1 << 23, 3000, gi.EINVAL), (1 << 24, 3000, gi.EUNSUPPORTED)):
        sizes = dict(B=8, D=D, L=L)
        if code == gi.EINVAL:
            sizes.update({"r_out.channel": 0})
        assert call("block_norm", **sizes) == code, (L, D)
    assert call("block_norm_backward", B=8, D=1500, L=1 << 23, **{"dr.channel": 0}) == gi.EINVAL
    assert call("block_norm", B=65535, D=64, L=1, **{"r_out.channel": 0, "r_out.batch": 0}) == gi.EINVAL


def test_generation_steps_of_large_batches(lib):  # noqa: F811
    """B*D < 2^24 is for forms whose grid runs over all rows; a step's does not."""
    for name in ("causal_conv_step", "state_scan_step"):
        for B, D, code in ((4096, 4096, gi.EINVAL), (2048, 8192, gi.EINVAL), (65535, 4000, gi.EINVAL),
                           (65535, 4100, gi.EUNSUPPORTED), (1, 1 << 24, gi.EUNSUPPORTED), (1, (1 << 24) - 2, gi.EINVAL),
                           (0, 4, gi.EINVAL)):
            sizes = dict(B=B, D=D, lines=65535)
            if code == gi.EINVAL:
                sizes.update(APART, **{"y.batch": 0})
            assert call(name, **sizes) == code, (name, B, D)
