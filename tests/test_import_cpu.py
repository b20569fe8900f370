"""The package without torch: the library's path, its loading, its structures
and the calls that take no tensor."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None  # an import of it raises ImportError
import grouped_query_kv_gb300 as g
assert g.library_path().endswith(".so")
assert g.lib().kvattn_status_string(0) == b"KVATTN_OK"
assert g.get_plan(8, 48, 1, 256, 32768, num_sms=152)["num_ctas"] == 152
g.set_tuning(0, 0)
try:
    g.kv_append(None, None, None, None, None)
except ImportError:
    print("torch wanted by the first tensor")
"""


def test_the_library_is_reached_without_torch():
    from grouped_query_kv_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "first tensor" in r.stdout


def test_torch_is_imported_once_at_the_first_tensor():
    code = ("import sys, grouped_query_kv_gb300 as g\n"
            "assert 'torch' not in sys.modules\n"
            "try:\n    g.kv_append(1, 2, 3, 4, 5)\n"
            "except TypeError:\n    pass\n"
            "import torch\n"
            "assert g.torch is torch\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
