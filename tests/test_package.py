"""What the package offers by name, no GPU: nothing is loaded before it is asked for."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_names():
    code = """
import sys
import tensor_adamw_optimizer_amd as t
assert "torch" not in sys.modules
assert set(t.__all__) == {"AdamW", "ApexwError", "_lib", "ops"}
assert callable(t.ops.gated_ffn) and callable(t.ops.linear_cross_entropy)
assert callable(t.ops.qk_norm_rope) and t.AdamW.__module__ == t.__name__ + ".optim"
assert t._lib._lib is None
try:
    t.nothing
except AttributeError as e:
    assert "nothing" in str(e)
else:
    raise SystemExit("a name that is not there was found")
"""
    subprocess.check_call([sys.executable, "-c", code], cwd=ROOT)
