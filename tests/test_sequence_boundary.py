"""Host-side tests of the sequence operators' C entry points: every bad argument
is refused before any HIP call (the fake pointers are never touched).  No test
here launches a kernel, so they run without a GPU.
"""
import ctypes
import os
import re
import struct

import pytest

import conv2d_backward_amd as gi

torch = pytest.importorskip("torch")
from conv2d_backward_amd import sequence  # noqa: E402

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "sequence_ops.h")
P = 0x1000  # a pointer that must not be followed


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gi.library_path):
        from conv2d_backward_amd import build
        build.build()
    return gi.load_library()


def fields_of(name):
    """The fields of an argument struct in sequence_ops.h, tensors as three."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s_args \{(.*?)\}" % name, text, re.S).group(1)
    out = []
    for line in body.split(";"):
        words = line.replace("*", " ").replace("const ", " ").split(None, 1)
        if len(words) == 2:
            for field in words[1].split(","):
                f = field.strip()
                out += [f, f + ".batch", f + ".channel"] if words[0] == "seq_tensor" else [f]
    return out


def format_of(name):
    """The struct format of an argument struct: its int32 and float fields, then 8-byte ones."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s_args \{(.*?)\}" % name, text, re.S).group(1)
    small = re.findall(r"\b(int32_t|float) ([^;*]*);", body)
    kinds = "".join(("i" if t == "int32_t" else "f") * len(names.split(",")) for t, names in small)
    return struct.Struct(kinds + "%dq" % (len(fields_of(name)) - len(kinds)))


STRUCTS = {n: format_of(n) for n in ("causal_conv", "causal_conv_backward", "causal_conv_step", "state_scan",
                                     "state_scan_backward", "state_scan_step", "block_norm",
                                     "block_norm_backward")}
ENTRIES = {"causal_conv": "causal_conv_forward", "state_scan": "state_scan_forward",
           "block_norm": "block_norm_forward"}
SIZES = {"B": 2, "D": 4, "L": 10, "K": 4, "N": 3, "G": 2, "lines": 2, "dtype": 0, "eps": 1e-6,
         "workspace_bytes": 1 << 20, "reserved": 0, "silu": 1, "softplus": 1}


def call(name, **change):
    values = []
    for f in fields_of(name):
        v = SIZES.get(f, P)
        if f.endswith(".batch"):
            v = 4 * 10
        if f.endswith(".channel"):
            v = 10
        values.append(change.get(f, v))
    return getattr(gi.load_library(), ENTRIES.get(name, name))(STRUCTS[name].pack(*values), None)


def workspace(name, *sizes):
    fn = getattr(gi.load_library(), name)
    fn.restype = ctypes.c_int64
    return fn(*sizes)


def test_binding_describes_the_structs(lib):
    """The binding's operands are the fields of the header's structs, in order."""
    for name in STRUCTS:
        header, _, scratch, operands = sequence._ENTRIES[ENTRIES.get(name, name)]
        fields = [f for f in fields_of(name) if "." not in f]
        sizes = header.split()
        assert len(fields) == 1 + len(sizes) + len(operands) + (2 if scratch else 0), name
        for f, s in zip(fields[1:], sizes):
            assert f == s, name
        wide = {f.split(".")[0] for f in fields_of(name) if "." in f}
        for f, o in zip(fields[1 + len(sizes):], operands):
            assert (f in wide) == (o[1] in (sequence._ACT, sequence._ACT32, sequence._STATES)), (name, f)


NEEDED = {
    "causal_conv": ("x", "y", "w"), "causal_conv_backward": ("gy", "x", "w"),
    "causal_conv_step": ("x", "y", "w", "state"),
    "state_scan": ("x", "dt", "Bm", "Cm", "y", "A"),
    "state_scan_backward": ("gout", "x", "dt", "Bm", "Cm", "dx", "ddt", "A", "checkpoints", "dBm",
                            "dCm", "dA", "workspace", "z", "dz"),
    "state_scan_step": ("x", "dt", "Bm", "Cm", "y", "A", "state"),
    "block_norm": ("y", "r", "r_out", "u", "w_pre"),
    "block_norm_backward": ("y", "r_out", "dy", "dr", "workspace", "scale", "w_post", "w_pre", "gate",
                            "dgate"),
}


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_refuses_null_pointers(lib, name):
    for field in NEEDED[name]:
        assert call(name, **{field: 0}) == gi.EINVAL, field


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_refuses_sizes_and_types(lib, name):
    fields = fields_of(name)
    for field in ("B", "D", "L", "K", "N", "G", "lines"):
        if field in fields:
            for v in (0, -1):
                assert call(name, **{field: v}) == gi.EINVAL, (field, v)
    for v in (-1, 3):
        assert call(name, dtype=v) == gi.EINVAL
    if "G" in fields:
        assert call(name, G=3) == gi.EINVAL          # does not divide D
        assert call(name, N=257) == gi.EUNSUPPORTED
    if "K" in fields:
        assert call(name, K=9) == gi.EUNSUPPORTED
    if "eps" in fields:
        for v in (-1.0, float("nan")):
            assert call(name, eps=v) == gi.EINVAL
    assert call(name, B=70000) == gi.EUNSUPPORTED
    assert call(name, B=1000, D=1 << 20) == gi.EUNSUPPORTED
    if "L" in fields:
        assert call(name, L=(1 << 26) + 1) == gi.EUNSUPPORTED
    if "lines" in fields:
        assert call(name, slots=0, lines=1) == gi.EINVAL   # fewer lines than rows


@pytest.mark.parametrize("name", sorted(n for n in STRUCTS if "L" in fields_of(n)))
def test_refuses_more_positions_than_a_grid_has(lib, name):
    assert call(name, B=32, L=1 << 26) == gi.EUNSUPPORTED
    if name.startswith("block_norm"):
        assert call(name, B=8, L=1 << 24) == gi.EUNSUPPORTED
        assert lib.block_norm_workspace(8, 4, 1 << 24, 1) == -1 < lib.block_norm_workspace(8, 4, 1 << 23, 1)


OUTPUTS = {"causal_conv": ("y",), "causal_conv_backward": ("dx",), "causal_conv_step": ("y",),
           "state_scan": ("y",), "state_scan_backward": ("dx", "ddt", "dz"), "state_scan_step": ("y",),
           "block_norm": ("r_out", "u"), "block_norm_backward": ("dy", "dr", "dgate")}


@pytest.mark.parametrize("name", sorted(STRUCTS))
def test_refuses_outputs_that_share_elements(lib, name):
    for out in OUTPUTS[name]:
        assert call(name, **{out + ".channel": 0}) == gi.EINVAL
        assert call(name, **{out + ".batch": 0}) == gi.EINVAL
        if "L" in fields_of(name):
            assert call(name, **{out + ".channel": 9}) == gi.EINVAL   # rows of 10 positions
            assert call(name, **{out + ".batch": 39}) == gi.EINVAL    # items of 4 rows


@pytest.mark.parametrize("name", ["state_scan_backward", "block_norm_backward"])
def test_refuses_workspaces(lib, name):
    assert call(name, workspace_bytes=16) == gi.EINVAL
    assert call(name, workspace=P + 4) == gi.EINVAL


def test_workspace_sizes(lib):
    assert workspace("causal_conv_workspace", 2, 4, 10, 4) >= 0
    assert workspace("state_scan_workspace", 2, 4, 10, 3, 2) > 0
    assert workspace("block_norm_workspace", 2, 4, 10, 1) > 0
    # invalid sizes
    assert workspace("causal_conv_workspace", 2, 4, 10, 9) == -1
    assert workspace("state_scan_workspace", 2, 4, 10, 3, 3) == -1
    assert workspace("block_norm_workspace", 2, 0, 10, 1) == -1


def test_gate_and_gradient_come_together(lib):
    assert call("block_norm_backward", gate=0) == gi.EINVAL
    assert call("block_norm", w_pre=0) == gi.EINVAL
    assert call("block_norm", u=0) == gi.EINVAL


def test_nothing_asked_is_nothing_done(lib):
    assert call("causal_conv_backward", dx=0, dw=0, db=0) == gi.OK


@pytest.mark.parametrize("call_", [
    lambda t: gi.causal_conv(t, torch.zeros(4, 2)),
    lambda t: gi.causal_conv_step(t[..., 0], torch.zeros(2, 4, 1), torch.zeros(4, 2)),
    lambda t: gi.state_scan(t, t, torch.zeros(4, 3), torch.zeros(2, 3, 5), torch.zeros(2, 3, 5)),
    lambda t: gi.block_norm(t, t),
])
def test_binding_rejects_cpu_tensors(lib, call_):
    with pytest.raises(ValueError):
        call_(torch.zeros(2, 4, 5))


def test_unknown_name_of_the_package():
    with pytest.raises(AttributeError):
        gi.no_such_operator
