"""Plans that just fit the library's own workspace: 8 MiB of work list,
counters and partial states, the requests' lengths not counted."""
import numpy as np
import pytest
import torch

LIMIT = 8 << 20


def _plan(C, batch, rope_theta=0.0):
    problem = C.make_problem(batch=batch, num_qo_heads=1, num_kv_heads=1, page_size=1, dtype="f16",
                             sm_scale=1.0, num_sms=148, ctas_per_sm=4, num_pages=256,
                             rope_theta=rope_theta)
    return C.pa_plan_create(problem, np.arange(batch + 1), np.ones(batch, np.int32))


def _lengths(batch):
    return -(-4 * batch // 256) * 256


def _largest(C):
    """The largest batch of one-token requests whose workspace without the
    lengths is at most 8 MiB."""
    lo, hi = 100_000, 300_000
    while hi - lo > 1:
        mid = (lo + hi) // 2
        if C.pa_plan_workspace_bytes(_plan(C, mid)) - _lengths(mid) <= LIMIT:
            lo = mid
        else:
            hi = mid
    return lo


def test_plans_that_fit_are_taken_and_others_refused():
    """Decided on the host: a plan that fits is refused by nothing but, where
    there is no GPU, the CUDA runtime."""
    from serving_attention_paged_b200 import pagedattn as C
    n = _largest(C)
    assert C.pa_plan_workspace_bytes(_plan(C, n)) > LIMIT
    for batch, rope_theta in ((n + 1, 0.0), (n, 1e4)):  # rotary runs read the lengths
        with pytest.raises(C.PagedAttnError) as e:
            C.pa_run_static_workspace(_plan(C, batch, rope_theta), *[1 << 20] * 5, None, 0)
        assert e.value.status == C.PA_ERR_WORKSPACE_TOO_SMALL
    if not torch.cuda.is_available():
        with pytest.raises(C.PagedAttnError) as e:
            C.pa_run_static_workspace(_plan(C, n), *[1 << 20] * 5, None, 0)
        assert e.value.status == C.PA_ERR_CUDA


@pytest.mark.gpu
def test_largest_plan_runs():
    """One token per request: o is its value, lse its score."""
    from serving_attention_paged_b200 import pagedattn as C
    n = _largest(C)
    plan = _plan(C, n)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(256, 1, 1, 128, generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn(n, 1, 128, generator=g, device="cuda").half() / 16
    pages = torch.randint(256, (n,), generator=g, device="cuda", dtype=torch.int32)
    o, lse = torch.full_like(q, 9.0), torch.full((n, 1), 9.0, device="cuda")
    C.pa_run_static_workspace(plan, q, k, v, pages, o, lse)
    torch.cuda.synchronize()
    assert C.pa_static_workspace_check(plan) == -1
    at = pages.long()
    # one weight of 1: only P's and o's rounding to fp16
    assert ((o - v[at, 0]).abs() <= v[at, 0].abs() * 2.0 ** -10).all()
    ref = (q.double() * k[at, 0].double()).sum(-1)
    assert (lse - ref).abs().max() <= 1e-3
