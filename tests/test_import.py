"""The package loads without torch: the build and the C library's bindings need
none; only the calls that take tensors do."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys


class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("torch is not here")


sys.meta_path.insert(0, NoTorch())
import quantized_weight_q4_gb300 as q4
from quantized_weight_q4_gb300 import _build
assert q4.library_path() == _build.LIB_PATH
assert q4.KvCacheStruct and q4.Q4_ROPE_PAIRS == 1
assert "KVCache" in dir(q4) and "q4_sample" in dir(q4)
try:
    q4.KVCache
    raise SystemExit("KVCache without torch")
except ImportError:
    pass
try:
    q4.no_such_name
    raise SystemExit("a name that is not there")
except AttributeError:
    pass
"""


def test_package_loads_without_torch():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr or r.stdout


def test_serving_names_are_the_package_s():
    import quantized_weight_q4_gb300 as q4
    from quantized_weight_q4_gb300 import serving
    for name in ("KVCache", "q4_kv_append", "q4_kv_gather", "q4_kv_attention", "q4_kv_attention_workspace_size",
                 "q4_sample"):
        assert getattr(q4, name) is getattr(serving, name)
