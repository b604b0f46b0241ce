"""The package where torch is not installed: it loads, and so does the library; only calls need torch."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None
from vision_transformer_attention_psapackqkv_gb300 import _build, binding
_build.build()
assert binding.load().psa_attention_bwd_workspace_size(binding.PsaShape(1, 2, 32, 8, 8, binding.PSA_DTYPE_BF16)) > 0
assert binding.psa_kv_evict_workspace_size(binding.PsaEvict(1, 1, 16, 64, binding.PSA_DTYPE_BF16, 8, 0, 0)) > 0
"""


def test_the_package_loads_without_torch():
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr
