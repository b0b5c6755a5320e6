"""What the package needs to be imported and to run the calls on quantised
weights: the library, and neither torch (until a call without a stream asks
for the current one) nor the 16-bit calls' helper.  CPU only."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = f"""
import sys
sys.path.insert(0, {ROOT!r})
class Missing:
    def find_spec(self, name, path=None, target=None):
        if name in ABSENT:
            raise ModuleNotFoundError("no module named " + name)
sys.meta_path.insert(0, Missing())
import quantized_moe_route_b200 as moe
"""


def run(absent, code):
    out = subprocess.run([sys.executable, "-c", f"ABSENT = {absent!r}\n{WITHOUT}\n{code}"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]


@pytest.mark.parametrize("absent", [["torch"], ["quantized_moe_route_b200._call"], ["torch", "quantized_moe_route_b200._call"]])
def test_quantised_calls_need_neither_torch_nor_the_helper(absent):
    run(absent, """
assert moe.moe_w4_packed_bytes(1024, 2048) == 1179648
assert moe.lib().moe_route(None, -1, 8, 2, None, None, None) == moe.MOE_ERR_INVALID_ARG
layer = moe.moe_w4_layer(8, 128, 64, 1 << 20, 1 << 20)
try:
    moe._check(moe.lib().moe_ffn_w4a16_decode(layer, None, None, -1, 2, None, None, 0, None), "decode")
except moe.MoeError as e:
    assert e.status == moe.MOE_ERR_INVALID_ARG
else:
    raise AssertionError
assert moe._stream(0) == 0
assert "torch" in ABSENT or "torch" not in sys.modules
""")


def test_16_bit_calls_say_that_the_helper_is_missing():
    run(["quantized_moe_route_b200._call"], """
try:
    moe._run("moe_linear", 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
except ImportError as e:
    assert "build.py" in str(e)
else:
    raise AssertionError
""")


def test_build_makes_the_library_before_the_helper(monkeypatch):
    """A machine without gcc or Python's headers still gets the library."""
    from quantized_moe_route_b200 import build
    made = []
    monkeypatch.setattr(build, "needs_build", lambda: True)
    monkeypatch.setattr(build, "build_call", lambda force=False: made.append("helper"))
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    monkeypatch.setattr(build.subprocess, "check_call", lambda cmd: made.append("library" if build.LIB in cmd[cmd.index("-o") + 1] else "?"))
    assert build.build() == build.LIB
    assert made == ["library", "helper"]
