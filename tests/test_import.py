"""The package is imported, inspected and star-imported without torch and without its
built extension module; only a call needs them.  Each case in a fresh interpreter."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys
class Refuse:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError("no torch here", name=name)
if %r:
    sys.meta_path.insert(0, Refuse())
"""

INSPECT = """
from conv2d_backward_amd import *
import conv2d_backward_amd as gi
assert "torch" not in sys.modules
for name in gi.__all__:
    assert hasattr(gi, name), name
    assert globals()[name] is getattr(gi, name)
assert set(gi.__all__) <= set(dir(gi)) and not hasattr(gi, "no_such_operator")
assert gi.SCAN_CHECKPOINT == 128 and gi.NormGrads._fields[0] == "dy"
"""


def run(text, without_torch):
    r = subprocess.run([sys.executable, "-c", SETUP % without_torch + text], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_star_import_without_torch():
    run(INSPECT, True)


def test_call_without_torch_says_so():
    run(INSPECT + """
gi.sequence._binding_path = gi.__file__   # (is there, and not loaded before torch)
try:
    causal_conv(None, None)
except ModuleNotFoundError as e:
    assert e.name == "torch"
else:
    raise AssertionError("not refused")
""", True)


def test_star_import_without_the_extension_module():
    run(INSPECT + """
gi.sequence._binding_path += ".missing"
for f in (lambda: causal_conv(None, None), lambda: block_norm(None, None)):
    try:
        f()
    except LibraryNotBuilt as e:
        assert "_sequence.so.missing" in str(e)
    else:
        raise AssertionError("not refused")
""", False)
