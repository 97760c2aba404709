"""The ctypes binding as a caller without torch uses it, and the C entries'
checks of addresses; no GPU."""
import os
import subprocess
import sys

import pytest

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


@pytest.mark.parametrize("name", ["k_scales", "v_scales", "kv_indices", "out_indices"])
def test_cache_calls_refuse_misaligned_scales_and_indices(name):
    """A 4-byte array at an odd address would fault on the device."""
    from serving_attention_paged_b200 import pagedattn as C
    problem = C.make_problem(batch=2, num_qo_heads=2, num_kv_heads=2, page_size=16, dtype="f16",
                             sm_scale=1.0, num_sms=1, ctas_per_sm=1, num_pages=64, kv_dtype="e4m3")
    plan = C.pa_kv_plan_create(problem, 16, [0, 3, 23], [0, 1, 3], [5, 4])
    a = 1 << 20
    args = dict(k=a, k_stride=256, v=a, v_stride=256, k_pool=a, v_pool=a, k_scales=a, v_scales=a,
                kv_indices=a, workspace=a, workspace_bytes=C.pa_plan_workspace_bytes(plan))
    calls = [lambda **kw: C.pa_kv_read(plan, **{**args, "out_indices": a, "num_out_pages": 4, **kw},
                                       stream=0)]
    if name != "out_indices":
        calls.append(lambda **kw: C.pa_kv_append(plan, **{**args, **kw}, stream=0))
    for call in calls:
        for off in (1, 2):
            with pytest.raises(C.PagedAttnError) as e:
                call(**{name: a + off})
            assert e.value.status == C.PA_ERR_INVALID_ARG
