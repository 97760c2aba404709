"""The ctypes binding as a caller without torch uses it, and the C entries'
checks of addresses; no GPU."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_binding_works_without_torch():
    """Plain addresses and stream handles need no torch, and do not load it."""
    code = """
import sys
sys.modules["torch"] = None  # importing it raises ImportError
from serving_attention_paged_b200 import pagedattn as C
p = C.make_problem(batch=1, num_qo_heads=8, num_kv_heads=2, page_size=16, dtype="f16",
                   sm_scale=0.1, num_sms=148, ctas_per_sm=1, num_pages=8)
plan = C.pa_plan_create(p, [0, 2], [5])
try:
    C.pa_run(plan, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20, None, 1 << 20, 0, 0)
except C.PagedAttnError as e:
    assert e.status == C.PA_ERR_WORKSPACE_TOO_SMALL
else:
    raise AssertionError("no refusal")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
