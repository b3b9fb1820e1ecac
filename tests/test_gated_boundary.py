"""Host-side tests of the C entry points of the gated recurrence and the 8-bit
projections: bad arguments are refused before any HIP call (the fake pointers are never
touched).  No test here launches a kernel.
"""
import ctypes

import pytest

import conv2d_backward_amd as gi
from conv2d_backward_amd import sequence
from test_sequence_boundary import P, fields_of, format_of, lib, workspace  # noqa: F401  (lib: a fixture)

torch = pytest.importorskip("torch")

NAMES = ("gated_scan", "gated_scan_backward", "gated_scan_step", "quantize_tokens", "project_int8", "project_int8_step")
ENTRIES = {"gated_scan": "gated_scan_forward"}
SIZES = {"B": 2, "D": 4, "E": 4, "L": 10, "K": 128, "lines": 2, "dtype": 0, "workspace_bytes": 1 << 20, "reserved": 0}


def call(name, **change):
    values = []
    for f in fields_of(name):
        v = SIZES.get(f, P)
        if f.endswith(".batch"):
            v = 4 * 10
        if f.endswith(".channel"):
            v = 10
        values.append(change.get(f, v))
    return getattr(gi.load_library(), ENTRIES.get(name, name))(format_of(name).pack(*values), None)


def test_binding_describes_the_structs(lib):  # noqa: F811
    for name in NAMES:
        header, _, scratch, operands = sequence._ENTRIES[ENTRIES.get(name, name)]
        fields = [f for f in fields_of(name) if "." not in f]
        sizes = header.split()
        assert len(fields) == 1 + len(sizes) + len(operands) + (2 if scratch else 0), name
        assert fields[1:1 + len(sizes)] == sizes, name
        wide = {f.split(".")[0] for f in fields_of(name) if "." in f}
        for f, o in zip(fields[1 + len(sizes):], operands):
            assert (f in wide) == (o[1] == sequence._ACT), (name, f)


NEEDED = {"gated_scan": "x r i A y", "gated_scan_backward": "gout x r i A dx dr di dA checkpoints workspace z dz",
          "gated_scan_step": "x r i A y state", "quantize_tokens": "x codes scales",
          "project_int8": "codes scales w w_scales y", "project_int8_step": "x w w_scales y workspace"}


@pytest.mark.parametrize("name", NAMES)
def test_refuses_null_pointers(lib, name):  # noqa: F811
    sizes = {"B": 40} if "workspace" in NEEDED[name] else {}   # (few rows need no workspace)
    for field in NEEDED[name].split():
        assert call(name, **{field: 0}, **sizes) == gi.EINVAL, field


@pytest.mark.parametrize("name", NAMES)
def test_refuses_sizes_and_types(lib, name):  # noqa: F811
    fields = fields_of(name)
    for field in ("B", "D", "E", "L", "K", "lines"):
        if field in fields:
            for v in (0, -1):
                assert call(name, **{field: v}) == gi.EINVAL, (field, v)
    for v in (-1, 3):
        assert call(name, dtype=v) == gi.EINVAL
    if "lines" in fields:
        assert call(name, slots=0, lines=1) == gi.EINVAL   # fewer lines than rows
    if "K" in fields:
        for v in (64, 127, 192, 1 << 30):
            assert call(name, K=v) in (gi.EINVAL, gi.EUNSUPPORTED), v
        for field in ("codes", "w"):
            if field in fields:
                assert call(name, **{field: P + 8}) == gi.EINVAL   # not on 16 bytes


def test_limits(lib):  # noqa: F811
    for name in NAMES[:3]:
        assert call(name, B=70000, lines=70000) == gi.EUNSUPPORTED
        assert call(name, B=2000, D=1 << 20, lines=2000) == gi.EUNSUPPORTED
    for name in NAMES[:2]:
        assert call(name, L=(1 << 26) + 1) == gi.EUNSUPPORTED
        assert call(name, B=32, L=1 << 26) == gi.EUNSUPPORTED
    apart = {"y.channel": 0}   # EINVAL, after the sizes
    assert call("gated_scan", B=1, D=(1 << 24) - 1, L=1 << 26, **apart) == gi.EINVAL
    assert call("gated_scan_step", B=65535, D=4000, lines=65535, **apart) == gi.EINVAL
    assert call("quantize_tokens", D=65537, K=65664) == gi.EUNSUPPORTED
    assert call("quantize_tokens", B=1 << 13, L=1 << 10) == gi.EUNSUPPORTED
    assert call("quantize_tokens", K=256) == gi.EINVAL          # not D rounded up
    assert call("project_int8", K=65664) == gi.EUNSUPPORTED
    assert call("project_int8", B=1 << 13, L=1 << 10) == gi.EUNSUPPORTED
    assert call("project_int8", E=1 << 24) == gi.EUNSUPPORTED
    assert call("project_int8", B=1, E=1 << 20, L=1 << 15) == gi.EUNSUPPORTED
    assert call("project_int8", B=1, E=1 << 20, L=1 << 14, **apart) == gi.EINVAL
    assert call("project_int8_step", D=65537, K=65664) == gi.EUNSUPPORTED
    assert call("project_int8_step", B=1 << 13, E=1 << 22) == gi.EUNSUPPORTED


def test_refuses_outputs_that_share_elements(lib):  # noqa: F811
    for name, outs in (("gated_scan", ["y"]), ("gated_scan_backward", ["dx", "dr", "di", "dz"]),
                       ("gated_scan_step", ["y"]), ("project_int8", ["y"]), ("project_int8_step", ["y"])):
        for out in outs:
            assert call(name, **{out + ".channel": 0}) == gi.EINVAL
            assert call(name, **{out + ".batch": 0}) == gi.EINVAL
            if "L" in fields_of(name):
                assert call(name, **{out + ".channel": 9}) == gi.EINVAL   # rows of 10 positions
                assert call(name, **{out + ".batch": 39}) == gi.EINVAL    # items of 4 rows


def test_workspaces(lib):  # noqa: F811
    for name in ("gated_scan_backward", "project_int8_step"):
        assert call(name, workspace_bytes=16, B=40) == gi.EINVAL
        assert call(name, workspace=P + 4, B=40) == gi.EINVAL
    assert workspace("gated_scan_workspace", 2, 4, 10) == 0 < workspace("gated_scan_workspace", 40, 4, 10)
    assert workspace("gated_scan_workspace", 2, 0, 10) == -1
    assert workspace("project_int8_step_workspace", 2, 4, 10) == 0 < workspace("project_int8_step_workspace", 40, 4, 10)
    assert workspace("project_int8_step_workspace", 2, 70000, 10) == -1


def test_gradients_of_what_is_not_there(lib):  # noqa: F811
    assert call("gated_scan_backward", r_bias=0) == gi.EINVAL
    assert call("gated_scan_backward", i_bias=0) == gi.EINVAL
    assert call("gated_scan_backward", z=0) == gi.EINVAL


def test_plans(lib):  # noqa: F811
    with pytest.raises(gi.Conv2dGiError):
        gi.gated_scan_plan(1, 0, 10)
    assert "lanes=" in gi.gated_scan_plan(2, 64, 10) and "waves=" in gi.gated_scan_plan(1, 4, 9000, True)
    buf = ctypes.create_string_buffer(4)
    assert gi.load_library().gated_scan_plan(2, 64, 10, 0, buf, 4) == gi.OK and len(buf.value) == 3
    assert gi.load_library().gated_scan_plan(2, 64, 10, 0, None, 4) == gi.EINVAL


@pytest.mark.parametrize("call_", [
    lambda t: gi.gated_scan(t, t, t, torch.zeros(4)),
    lambda t: gi.gated_scan_step(t[..., 0], t[..., 0], t[..., 0], torch.zeros(4), torch.zeros(2, 4)),
    lambda t: gi.quantize_tokens(t), lambda t: gi.quantize_weight(t[0]),
    lambda t: gi.project_int8(torch.zeros(2, 5, 128, dtype=torch.int8), torch.zeros(2, 5),
                              torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)),
    lambda t: gi.project_int8_step(t[..., 0], torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4)),
])
def test_binding_rejects_cpu_tensors(lib, call_):  # noqa: F811
    with pytest.raises(ValueError):
        call_(torch.zeros(2, 4, 5))
