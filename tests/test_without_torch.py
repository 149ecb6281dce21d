"""The host parts of the package work where torch is not installed."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BODY = """
import sys
sys.modules["torch"] = None  # importing it fails
import ternary_quantized_gemv_amd as bq
assert bq.bq_packed_bytes(bq.BQ_Q1_0, 64, 128) == (1024, 1024)
from ternary_quantized_gemv_amd.staging import chain_groups
assert len(chain_groups(2)) == 9
print("ok")
"""


def test_host_calls_without_torch():
    r = subprocess.run([sys.executable, "-c", BODY], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
