"""The fp64 definitions of the block-scaled cache and of capped, biased
attention, pinned by torch's FP8 conversion, closed forms, the plain oracle
and hand-worked blocks; and the argument checks of the C entry points (they
happen before any CUDA call)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache
from serving_attention_paged_b200 import workloads as W

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


@pytest.fixture(scope="module")
def C():
    from serving_attention_paged_b200 import build
    build.build()
    from serving_attention_paged_b200 import pagedattn
    return pagedattn


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_encode_matches_torch_and_is_idempotent(fmt):
    """Random values, every code's value, every midpoint of neighbours."""
    v = cache.fp8_table(fmt)
    fine = np.sort(v[np.isfinite(v)])
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 100,
                        np.random.default_rng(1).standard_normal(20000) * 1e-3,
                        fine, (fine[1:] + fine[:-1]) / 2])
    x = x[np.abs(x) <= cache.FP8_MAX[fmt]].astype(np.float32)
    ref = torch.from_numpy(x).to(FP8[fmt]).view(torch.uint8).numpy()
    got = cache.fp8_encode(x, fmt)
    assert np.array_equal(v[got], v[ref])
    assert np.array_equal(cache.fp8_encode(fine, fmt)[fine != 0],
                          cache.fp8_encode(v[cache.fp8_encode(fine, fmt)], fmt)[fine != 0])
    big = cache.fp8_encode([1e30, -np.inf, np.nan], fmt)
    assert v[big[0]] == cache.FP8_MAX[fmt] and v[big[1]] == -cache.FP8_MAX[fmt]
    assert np.isnan(v[big[2]])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_scale_is_the_smallest_power_of_two(fmt):
    top = cache.FP8_MAX[fmt]
    for e in (-40, -7, 0, 9, 30):
        s = 2.0 ** e
        assert cache.scale_for(top * s, fmt) == s
        assert cache.scale_for(np.nextafter(top * s, np.inf), fmt) == 2 * s
        assert cache.scale_for(top * s / 2, fmt) == s / 2
    assert cache.scale_for(0.0, fmt) == 2.0 ** -60
    assert cache.scale_for(1e38, fmt) == 2.0 ** 60


def test_append_by_hand():
    """One head, 4 elements, blocks of 4 tokens in pages of 4: a first token
    sets the scale whatever was there, a smaller one keeps it, a larger one
    moves the earlier codes."""
    codes = np.full((2, 4, 1, 4), 0x55, dtype=np.uint8)
    scales = np.array([[777.0], [3.0]])
    kw = dict(page_size=4, scale_block=4, dtype="f16", fmt="e4m3")
    first = torch.tensor([[[1.75, -0.875, 0.0, 7.0]]], dtype=torch.float16)
    c, s = cache.kv_append(first, codes, scales, [0, 1], [0, 1], [1], [1], **kw)
    assert s.tolist() == [[777.0], [2.0 ** -6]]  # 7 = 448 / 64
    assert cache.fp8_table("e4m3")[c[1, 0, 0]].tolist() == [112.0, -56.0, 0.0, 448.0]
    assert (c[0] == 0x55).all() and (c[1, 1:] == 0x55).all()  # nothing else is touched
    small = torch.tensor([[[0.015625, 0, 0, 0]]], dtype=torch.float16)
    c, s = cache.kv_append(small, c, s, [0, 1], [0, 1], [1], [2], **kw)
    assert s[1, 0] == 2.0 ** -6 and cache.fp8_table("e4m3")[c[1, 1, 0, 0]] == 1.0
    large = torch.tensor([[[56.0, 0, 0, 0]]], dtype=torch.float16)
    c, s = cache.kv_append(large, c, s, [0, 1], [0, 1], [1], [3], **kw)
    assert s[1, 0] == 2.0 ** -3
    assert cache.fp8_table("e4m3")[c[1, 0, 0]].tolist() == [14.0, -7.0, 0.0, 56.0]
    assert cache.fp8_table("e4m3")[c[1, 1, 0, 0]] == 0.125
    assert (c[1, 3] == 0x55).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_append_then_read_is_within_half_a_step(fmt):
    lens, P = [37, 1, 16, 90], 16
    indptr, indices, last = W.tables_from_lengths(lens, P, W.permutation(5, 12))
    qo = np.concatenate([[0], np.cumsum(lens)])
    x = torch.randn(sum(lens), 2, 128, generator=torch.Generator().manual_seed(3)).bfloat16()
    codes, scales = np.zeros((12, P, 2, 128), np.uint8), np.zeros((12, 2))
    c, s = cache.kv_append(x, codes, scales, qo, indptr, indices, last, page_size=P,
                           scale_block=P, dtype="bf16", fmt=fmt)
    back = cache.kv_read(c, s, indptr, indices, last, page_size=P, scale_block=P, dtype="bf16",
                         fmt=fmt)
    ref = x.double().numpy()
    tiny = s.max() * cache.fp8_table(fmt)[1]
    assert np.all(np.abs(back - ref) <= np.abs(ref) * (2.0 ** -4 if fmt == "e4m3" else 2.0 ** -3)
                  + tiny / 2)


def test_attention_agrees_with_the_plain_oracle():
    """Without options, with one scale per tensor, and with rotary positions."""
    for fmt, theta in ((None, 0.0), ("e4m3", 0.0), (None, 1e4)):
        w = W.make_workload("x", [0, 1, 17, 60], num_qo_heads=4, num_kv_heads=2, page_size=16,
                            dtype="f16", seed=5, kv_dtype=fmt, k_scale=0.37, v_scale=1.3)
        t = w.materialize()
        kw = dict(num_qo_heads=4, num_kv_heads=2, page_size=16, dtype="f16", sm_scale=w.sm_scale)
        o1, l1 = oracle.paged_decode(t["q"], t["k_pool"], t["v_pool"], w.kv_indptr, w.kv_indices,
                                     w.last_page_len, head_dim=128, kv_dtype=fmt, k_scale=0.37,
                                     v_scale=1.3, rope_theta=theta, **kw)
        o2, l2 = cache.attention(t["q"], t["k_pool"], t["v_pool"], w.kv_indptr, w.kv_indices,
                                 w.last_page_len, fmt=fmt, k_scale=0.37, v_scale=1.3,
                                 rope_theta=theta, **kw)
        assert np.abs(o1 - o2).max() < 1e-12
        assert np.array_equal(np.isneginf(l1), np.isneginf(l2))
        assert np.abs(l1[~np.isneginf(l1)] - l2[~np.isneginf(l2)]).max() < 1e-12


def test_attention_prefill_agrees_with_the_plain_oracle():
    w = W.make_workload("x", [70, 5], num_qo_heads=4, num_kv_heads=2, page_size=16, dtype="bf16",
                        seed=6, qo_lens=[20, 5])
    t = w.materialize()
    for causal in (True, False):
        args = (w.kv_indptr, w.kv_indices, w.last_page_len)
        kw = dict(num_qo_heads=4, num_kv_heads=2, page_size=16, dtype="bf16",
                  sm_scale=w.sm_scale, causal=causal)
        o1, l1 = oracle.paged_prefill(t["q"], t["k_pool"], t["v_pool"], w.qo_indptr, *args,
                                      head_dim=128, **kw)
        o2, l2 = cache.attention(t["q"], t["k_pool"], t["v_pool"], *args, qo_indptr=w.qo_indptr,
                                 **kw)
        assert np.abs(o1 - o2).max() < 1e-12 and np.abs(l1 - l2).max() < 1e-12


def test_capped_and_biased_scores_closed_forms():
    w = W.make_workload("x", [40], num_qo_heads=2, num_kv_heads=2, page_size=8, dtype="f16",
                        seed=7)
    t = w.materialize()
    args = (t["q"], t["k_pool"], t["v_pool"], w.kv_indptr, w.kv_indices, w.last_page_len)
    kw = dict(num_qo_heads=2, num_kv_heads=2, page_size=8, dtype="f16", sm_scale=w.sm_scale)
    plain = cache.attention(*args, **kw)
    # a huge cap changes nothing; a tiny one makes the scores equal
    assert np.abs(cache.attention(*args, logit_cap=1e6, **kw)[0] - plain[0]).max() < 1e-9
    flat = cache.attention(*args, logit_cap=1e-9, **kw)
    v = cache.cached_rows(t["v_pool"], cache._rows(0, w.kv_indptr, w.kv_indices, w.last_page_len, 8),
                          dtype="f16")
    assert np.abs(flat[0][0, 0] - v[:, 0].mean(0)).max() < 1e-6
    assert abs(flat[1][0, 0] - np.log(40)) < 1e-6
    # a steep slope leaves the last token alone; its bias is 0, so lse = s_last
    steep = cache.attention(*args, alibi_slopes=np.array([1e4, 0.0]), **kw)
    assert np.abs(steep[0][0, 0] - v[-1, 0]).max() < 1e-12
    assert np.abs(steep[0][0, 1] - plain[0][0, 1]).max() < 1e-12


def _kv_problem(C, **kw):
    base = dict(batch=2, num_qo_heads=2, num_kv_heads=2, page_size=16, dtype="f16", sm_scale=1.0,
                num_sms=1, ctas_per_sm=1, num_pages=8, kv_dtype="e4m3")
    return C.make_problem(**{**base, **kw})


def test_kv_plan_validation(C):
    qo, indptr, last = [0, 3, 23], [0, 1, 3], [5, 4]
    plan = C.pa_kv_plan_create(_kv_problem(C), 16, qo, indptr, last)
    assert C.pa_plan_workspace_bytes(plan) > 0 and not C.pa_plan_uses_tensor_cores(plan)

    def status(problem=None, block=16, qo=qo, indptr=indptr, last=last):
        with pytest.raises(C.PagedAttnError) as e:
            C.pa_kv_plan_create(problem or _kv_problem(C), block, qo, indptr, last)
        return e.value.status

    for block in (0, -1, 3, 32, 12):
        assert status(block=block) == C.PA_ERR_INVALID_ARG
    assert status(_kv_problem(C, kv_dtype="f16")) == C.PA_ERR_INVALID_ARG
    assert status(_kv_problem(C, k_scale=0.5)) == C.PA_ERR_INVALID_ARG
    assert status(_kv_problem(C, v_scale=2.0)) == C.PA_ERR_INVALID_ARG
    assert status(_kv_problem(C, page_size=12)) == C.PA_ERR_UNSUPPORTED
    assert status(_kv_problem(C, head_dim=64)) == C.PA_ERR_UNSUPPORTED
    assert status(qo=[0, 6, 23]) == C.PA_ERR_INVALID_ARG      # 6 new tokens of 5
    assert status(qo=[0, 3, 2]) == C.PA_ERR_INVALID_ARG       # decreasing
    assert status(qo=[1, 3, 23]) == C.PA_ERR_INVALID_ARG
    assert status(indptr=[0, 2, 1]) == C.PA_ERR_INVALID_ARG
    assert status(last=[17, 4]) == C.PA_ERR_INVALID_ARG
    assert status(last=[0, 4]) == C.PA_ERR_INVALID_ARG
    C.pa_kv_plan_create(_kv_problem(C, batch=0), 16, [0], [0], [])  # nothing to do is a plan


def test_kv_run_argument_checks(C):
    """Refusals happen on the host; the addresses are never read."""
    plan = C.pa_kv_plan_create(_kv_problem(C), 16, [0, 3, 23], [0, 1, 3], [5, 4])
    n, a, row = C.pa_plan_workspace_bytes(plan), 1 << 20, 256
    good = dict(k=a, k_stride=row, v=a, v_stride=row, k_pool=a, v_pool=a, k_scales=a, v_scales=a,
                kv_indices=a, workspace=a, workspace_bytes=n)

    def append(**kw):
        with pytest.raises(C.PagedAttnError) as e:
            C.pa_kv_append(plan, **{**good, **kw}, stream=0)
        return e.value.status

    def read(**kw):
        with pytest.raises(C.PagedAttnError) as e:
            C.pa_kv_read(plan, **{**good, "out_indices": None, "num_out_pages": 0, **kw},
                         stream=0)
        return e.value.status

    for call in (append, read):
        for name in ("k", "v", "k_pool", "v_pool", "k_scales", "v_scales", "kv_indices",
                     "workspace"):
            assert call(**{name: None}) == C.PA_ERR_INVALID_ARG, name
        for name in ("k", "v", "k_pool", "v_pool"):
            assert call(**{name: a + 8}) == C.PA_ERR_INVALID_ARG, name
        for stride in (row - 8, row + 4, 0, -row):
            assert call(k_stride=stride) == C.PA_ERR_INVALID_ARG
            assert call(v_stride=stride) == C.PA_ERR_INVALID_ARG
        assert call(workspace=a + 16) == C.PA_ERR_INVALID_ARG
        assert call(workspace_bytes=n - 1) == C.PA_ERR_WORKSPACE_TOO_SMALL
    assert read(out_indices=a, num_out_pages=4, k_stride=row + 8) == C.PA_ERR_INVALID_ARG
    assert read(out_indices=a, num_out_pages=-1) == C.PA_ERR_INVALID_ARG
    assert read(out_indices=a, num_out_pages=1 << 40) == C.PA_ERR_UNSUPPORTED
    # other plans, and cache plans elsewhere
    w = W.make_workload("v", [20, 40], num_qo_heads=2, num_kv_heads=2, page_size=16, dtype="f16",
                        seed=1)
    decode = C.pa_plan_create(_kv_problem(C), w.kv_indptr, w.last_page_len)
    with pytest.raises(C.PagedAttnError):
        C.pa_kv_append(decode, **{**good, "workspace_bytes": 1 << 30}, stream=0)
    for call in (C.pa_run, C.pa_prefill_run):
        with pytest.raises(C.PagedAttnError) as e:
            call(plan, a, a, a, a, a, None, a, n, 0)
        assert e.value.status == C.PA_ERR_INVALID_ARG
    with pytest.raises(C.PagedAttnError) as e:
        C.pa_cascade_run(plan, a, a, a, a, a, a, None, a, n, 0)
    assert e.value.status == C.PA_ERR_INVALID_ARG
    with pytest.raises(C.PagedAttnError) as e:
        C.pa_run_static_workspace(plan, a, a, a, a, a, None, 0)
    assert e.value.status == C.PA_ERR_INVALID_ARG
    # nothing to write: nothing is asked of the pointers
    idle = C.pa_kv_plan_create(_kv_problem(C), 16, [0, 0, 0], [0, 1, 3], [5, 4])
    C.pa_kv_append(idle, None, 0, None, 0, None, None, None, None, None, a,
                   C.pa_plan_workspace_bytes(idle), 0)


def test_option_checks(C):
    """Refused on the host, before anything is enqueued."""
    w = W.make_workload("v", [20, 40], num_qo_heads=8, num_kv_heads=2, page_size=16, dtype="f16",
                        seed=1, qo_lens=[4, 4])
    a, big = 1 << 20, 1 << 30

    def problem(**kw):
        return C.make_problem(**{**dict(batch=2, num_qo_heads=8, num_kv_heads=2, page_size=16,
                                        dtype="f16", sm_scale=0.1, num_sms=4, ctas_per_sm=1,
                                        num_pages=w.num_pages), **kw})

    def status(plan, run=None, **kw):
        with pytest.raises(C.PagedAttnError) as e:
            (run or C.pa_run_options)(plan, C.make_options(**kw), a, a, a, a, a, None, a, big, 0)
        return e.value.status

    tables = (w.kv_indptr, w.last_page_len)
    p16, p8 = C.pa_plan_create(problem(), *tables), C.pa_plan_create(problem(kv_dtype="e4m3"), *tables)
    scaled = dict(k_scales=a, v_scales=a, scale_block=16)
    assert status(p16, **scaled) == C.PA_ERR_INVALID_ARG               # 16-bit pools
    for kw in (dict(k_scales=None), dict(v_scales=None), dict(scale_block=0), dict(scale_block=-4),
               dict(scale_block=3), dict(scale_block=32), dict(k_scales=a + 2)):
        assert status(p8, **{**scaled, **kw}) == C.PA_ERR_INVALID_ARG, kw
    other = C.pa_plan_create(problem(kv_dtype="e4m3", k_scale=0.5), *tables)
    assert status(other, **scaled) == C.PA_ERR_INVALID_ARG             # two kinds of scales
    for cap in (-1.0, float("nan"), float("inf"), 2.0 ** 21, 2.0 ** -21):
        assert status(p16, logit_cap=cap) == C.PA_ERR_INVALID_ARG
    assert status(p16, alibi_slopes=a + 1) == C.PA_ERR_INVALID_ARG
    cascade = C.pa_cascade_plan_create(problem(), 32, *tables)
    assert status(cascade, logit_cap=1.0) == C.PA_ERR_INVALID_ARG
    pre = [C.pa_prefill_plan_create(problem(), causal, w.qo_indptr, *tables) for causal in (1, 0)]
    assert status(pre[0], logit_cap=1.0) == C.PA_ERR_INVALID_ARG       # not a decode plan
    assert status(p16, C.pa_prefill_run_options, logit_cap=1.0) == C.PA_ERR_INVALID_ARG
    assert status(pre[0], C.pa_prefill_run_options, **scaled) == C.PA_ERR_UNSUPPORTED
    assert status(pre[1], C.pa_prefill_run_options, alibi_slopes=a) == C.PA_ERR_UNSUPPORTED
    assert status(pre[1], C.pa_prefill_run_options, logit_cap=-2.0) == C.PA_ERR_INVALID_ARG
