"""Prefill with options where its arithmetic is at its limits."""
import numpy as np
import pytest
import torch

from oracle import cache
from parity import assert_close, to_np
from test_attention_options_gpu import Case
from test_small_weights_gpu import D, G, HALF, P, Tail, _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_tail_behind_a_sink(dtype, slopes):
    """Two new tokens at the end of 131,072: the sink takes 0.9 of the softmax,
    each other token 12.5 steps of fp16's smallest, 2^-24, of it.  Slopes of
    zero turn the order of the key tiles around."""
    from serving_attention_paged_b200.wrapper import PagedPrefill
    case = Tail(128, 12.5 * 2.0 ** -24, 0.0)
    indptr, last, indices = case.tables()
    pf = PagedPrefill([0, 2], indptr, last, num_qo_heads=G, num_kv_heads=1, page_size=P,
                      dtype=dtype, sm_scale=case.top, num_pages=2)
    k, v = (torch.from_numpy(x).to(HALF[dtype]).cuda() for x in case.pools())
    q = torch.zeros(2, G, D, dtype=HALF[dtype], device="cuda")
    q[..., 0] = 1.0
    # a cap of 2^20 leaves scores of this size as they are, to a part in 10^9
    o, lse = pf.run(q, k, v, torch.from_numpy(indices).cuda(), logit_cap=0.0 if slopes else 2.0 ** 20,
                    alibi_slopes=torch.zeros(G, device="cuda") if slopes else None)
    torch.cuda.synchronize()
    assert pf.check() == -1
    ref, ref_lse = case.expected()
    # (the first new token misses one of 131,072 tokens of the tail)
    _close((to_np(o), to_np(lse)), ref, ref_lse, dtype, str(slopes))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group,kv,new", [(1, 128, 256), (1, 0, 129), (2, 64, 128), (4, 96, 64),
                                          (4, 992, 64), (8, 112, 32)])
def test_values_of_later_tiles_do_not_reach_earlier_tokens(group, kv, new, dtype):
    """Infinities and NaN among the values of the last new tokens.  Tokens whose
    128-key tiles end before them (those of an item's first half, here) must
    not notice, with a distance bias as without."""
    from serving_attention_paged_b200.wrapper import PagedPrefill
    per_half = 128 // group
    length = kv + new
    c = Case([length], group, 8, dtype, seed=group + new, qo=[new])
    w = c.w
    rows = torch.from_numpy(cache._rows(0, w.kv_indptr, w.kv_indices, w.last_page_len, 8))
    # tokens of the first half see keys below kv + per_half
    edge = -(-(kv + per_half) // 128) * 128
    assert edge < length, "the case has a tile that the first half does not see"
    ref = c.expected(qo_indptr=w.qo_indptr, logit_cap=20.0, alibi_slopes=c.slopes)
    plain = c.expected(qo_indptr=w.qo_indptr)
    v = c.pools[1].view(-1, 2, D)
    v[rows[edge:], :, ::2] = float("inf")
    v[rows[edge:], :, 1::2] = float("nan")
    pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=w.num_qo_heads,
                      num_kv_heads=2, page_size=8, dtype=dtype, sm_scale=w.sm_scale,
                      num_pages=w.num_pages)
    n = min(per_half, new)
    for cap, slopes, want in ((0.0, False, plain), (20.0, True, ref)):
        o, lse = c.run(pf, cap, slopes)
        assert np.isfinite(o[:n]).all(), f"slopes={slopes}"
        assert_close(o[:n], lse[:n], want[0][:n], want[1][:n], dtype, f"slopes={slopes}")


def test_small_scores_under_a_cap_are_exact_to_fp32():
    """One key per token: lse is the capped score itself.  cap = 2^15,
    sm_scale = 1 and scores of 160 to 1,640 (up to a twentieth of the cap).
    Rounded constants common to all: log2 e and ln 2 (their product is within
    0.7 of 2^-24 of 1), the polynomial's first coefficient (1), so at most 1.7
    parts of 2^-24; the roundings of each score's own (product, exponent,
    log-sum, last product) are within 4, of either sign, and their mean over
    512 scores within 1.  (2^-24 = 6e-8.)  So the mean error is below 3 * 2^-24."""
    from serving_attention_paged_b200.wrapper import PagedPrefill
    n, cap = 512, 2.0 ** 15
    g = np.random.default_rng(5)
    s = g.uniform(0.005, 0.05, n) * cap
    for dtype in ("f16", "bf16"):
        a = torch.from_numpy(np.sqrt(s)).to(HALF[dtype])
        q = torch.zeros(n, 1, D, dtype=HALF[dtype])
        q[:, 0, 3] = a
        k = torch.zeros(n, 8, 1, D, dtype=HALF[dtype])
        k[:, 0, 0, 3] = a
        exact = cap * np.tanh(a.double().numpy() ** 2 / cap)
        pf = PagedPrefill(np.arange(n + 1), np.arange(n + 1), np.ones(n, np.int32), num_qo_heads=1,
                          num_kv_heads=1, page_size=8, dtype=dtype, sm_scale=1.0, num_pages=n)
        _, lse = pf.run(q.cuda(), k.cuda(), torch.zeros_like(k).cuda(),
                        torch.arange(n, dtype=torch.int32, device="cuda"), logit_cap=cap)
        off = to_np(lse)[:, 0] / exact - 1.0
        assert abs(off.mean()) <= 3 * 2.0 ** -24, dtype
        assert np.abs(off).max() <= 8 * 2.0 ** -24, dtype


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_appends_to_long_contexts(group, dtype):
    """70 new tokens behind 16,500 and 20,011, with steep, flat and no bias."""
    from serving_attention_paged_b200.wrapper import PagedPrefill
    c = Case([16570, 20011], group, 64, dtype, hkv=1, seed=31 + group, qo=[70, 33])
    w = c.w
    c.slopes = torch.tensor([0.5, 1e-4, 0.0, 0.01] * 2)[:group].clone()
    pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=group, num_kv_heads=1,
                      page_size=64, dtype=dtype, sm_scale=w.sm_scale, num_pages=w.num_pages)
    for cap, slopes in ((30.0, True), (3.0, False), (0.0, True)):
        got = c.run(pf, cap, slopes)
        ref = c.expected(qo_indptr=w.qo_indptr, logit_cap=cap,
                         alibi_slopes=c.slopes if slopes else None)
        assert np.isfinite(got[0]).all()
        assert_close(*got, *ref, dtype, f"G={group} cap={cap} {slopes}")
