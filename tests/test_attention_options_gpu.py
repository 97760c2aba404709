"""Decode and prefill with options on the GPU against the fp64 definition in
oracle/cache.py: 8-bit pools with block scales, scores capped by a tanh and
biased by distance, alone and together, on both decode kernels.

Tolerances are the library's (tests/parity.py): 2e-3 on o plus a half-ulp of
the output type where that is larger, 1e-3 on lse.  Cached values are kept
near 1, as in the other parity tests, or o's tolerance scales with the largest
|v| (the error of o is a weighted mean of errors of v's size).
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache
from parity import O_TOL, assert_close, half_ulp, to_np
from serving_attention_paged_b200 import workloads as W

pytestmark = pytest.mark.gpu

EDGE_LENS = [0, 1, 15, 16, 17, 31, 33, 100, 257, 1000]
KERNELS = {"cuda_cores": 2, "tensor_cores": 4}  # PA_FLAG_CUDA_CORES / PA_FLAG_TENSOR_CORES
SPLITS = (dict(num_sms=10000, ctas_per_sm=1), dict(num_sms=3, ctas_per_sm=1, min_chunk_tokens=16))


class Case:
    """A paged decode problem; with ``fmt`` its pools hold codes and scales."""

    def __init__(self, lens, G, P, dtype, fmt=None, block=0, hkv=2, seed=0, spread=2.0, qo=None):
        w = W.make_workload("options", lens, num_qo_heads=hkv * G, num_kv_heads=hkv, page_size=P,
                            dtype=dtype, seed=seed + 7 * G + P, extra_pages=3, qo_lens=qo)
        t = w.materialize()
        self.w, self.fmt, self.block, self.k_scales, self.v_scales = w, fmt, block, None, None
        self.q, self.pools = t["q"], [t["k_pool"], t["v_pool"]]
        if fmt:
            rng = np.random.default_rng(seed)
            scales = []
            for i, pool in enumerate(self.pools):
                x = cache._widen16(pool, dtype).reshape(-1, hkv, 128)
                n = x.shape[0] // block
                # scales that differ by up to 2^(2 spread) from block to block
                s = 2.0 ** rng.uniform(-spread, spread, (n, hkv)) / 64
                s = s.astype(np.float32).astype(np.float64)
                codes = cache.fp8_encode(x / np.repeat(s, block, axis=0)[..., None], fmt)
                self.pools[i] = torch.from_numpy(codes).view(pool.shape)
                scales.append(torch.from_numpy(s.astype(np.float32)))
            self.k_scales, self.v_scales = scales
        self.slopes = torch.from_numpy(
            (2.0 ** (-8.0 * np.arange(1, hkv * G + 1) / (hkv * G))).astype(np.float32))

    def expected(self, **kw):
        w = self.w
        return cache.attention(self.q, *self.pools, w.kv_indptr, w.kv_indices, w.last_page_len,
                               num_qo_heads=w.num_qo_heads, num_kv_heads=w.num_kv_heads,
                               page_size=w.page_size, dtype=w.dtype, sm_scale=w.sm_scale,
                               fmt=self.fmt, k_scales=self.k_scales, v_scales=self.v_scales,
                               scale_block=self.block, **kw)

    def plan(self, rope_theta=0.0, **kw):
        from serving_attention_paged_b200.wrapper import PagedDecode
        w = self.w
        return PagedDecode(w.kv_indptr, w.last_page_len, num_qo_heads=w.num_qo_heads,
                           num_kv_heads=w.num_kv_heads, page_size=w.page_size, dtype=w.dtype,
                           sm_scale=w.sm_scale, num_pages=w.num_pages, kv_dtype=self.fmt,
                           rope_theta=rope_theta, **kw)

    def run(self, pd, cap=0.0, slopes=False, **kw):
        options = dict(logit_cap=cap, alibi_slopes=self.slopes.cuda() if slopes else None)
        if self.fmt:
            options.update(k_scales=self.k_scales.cuda(), v_scales=self.v_scales.cuda(),
                           scale_block=self.block)
        o, lse = pd.run(self.q.cuda(), *[p.cuda() for p in self.pools],
                        torch.from_numpy(self.w.kv_indices).cuda(), **options, **kw)
        torch.cuda.synchronize()
        assert pd.check() == -1
        return to_np(o), to_np(lse)


def _close(got, ref, dtype, what, vmax=1.0):
    """The library's tolerance, o's scaled by the largest cached value."""
    if vmax <= 4.0:  # N(0, 1) values
        assert_close(*got, *ref, dtype, what)
        return
    o, lse = got
    empty = np.isneginf(ref[1])
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0), what
    assert np.all(np.abs(o - ref[0]) <= O_TOL * vmax / 4 + half_ulp(ref[0], dtype)), what
    assert np.all(np.abs(lse - ref[1])[~empty] <= 1e-3), what


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("P,block", [(1, 1), (16, 16), (16, 4), (64, 1), (64, 64)])
def test_block_scales(P, block, group, dtype, fmt, kernel):
    c = Case(EDGE_LENS, group, P, dtype, fmt, block, seed=P + block)
    ref = c.expected()
    for kw in SPLITS:
        pd = c.plan(flags=KERNELS[kernel], **kw)
        _close(c.run(pd), ref, dtype, f"{kernel} {fmt} G={group} P={P}/{block} {kw}")


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_cap_and_bias(group, dtype, fmt, kernel):
    c = Case(EDGE_LENS, group, 16, dtype, fmt, 8 if fmt else 0, seed=3)
    for cap, slopes in ((2.0, False), (30.0, True), (0.0, True), (1000.0, False)):
        ref = c.expected(logit_cap=cap, alibi_slopes=c.slopes if slopes else None)
        for kw in SPLITS:
            pd = c.plan(flags=KERNELS[kernel], **kw)
            _close(c.run(pd, cap, slopes), ref, dtype, f"{kernel} {fmt} cap={cap} {slopes} {kw}")


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_value_scales_over_a_wide_range(kernel):
    """V scales from 2^-40 to 2^20 in one request, the large ones on tokens
    whose weight is about 2^-50: o is carried by the small ones, and their
    weights must keep their precision."""
    P, L = 16, 256
    c = Case([L], 4, P, "bf16", "e4m3", P, seed=5, spread=0.5)
    w = c.w
    rows = cache._rows(0, w.kv_indptr, w.kv_indices, w.last_page_len, P)
    blocks = rows[::P] // P
    c.v_scales[blocks] = 2.0 ** -40
    c.v_scales[blocks[3]] = 0.0              # a block of zeros
    c.v_scales[blocks[5]] = 2.0 ** 20
    # keys of block 5: minus a large multiple of every q head's mean direction
    c.k_scales[blocks[5]] = 2.0 ** -3
    q = cache._widen16(c.q, "bf16").reshape(2, 4, 128)
    key = np.stack([np.linalg.pinv(q[h]) @ np.full(4, -60.0 * np.log(2) / w.sm_scale)
                    for h in range(2)])
    codes = cache.fp8_encode(key * 8.0, "e4m3")
    c.pools[0].view(-1, 2, 128)[torch.from_numpy(rows[5 * P:6 * P])] = torch.from_numpy(codes)
    ref = c.expected()
    pd = c.plan(flags=KERNELS[kernel], num_sms=10000, ctas_per_sm=1)
    o, lse = c.run(pd)
    # block 5 contributes 2^20 * 448 * 2^-50ish at most; the others 2^-40 * |c|
    assert np.all(np.abs(o - ref[0]) <= 2e-3 * np.abs(ref[0]).max() + half_ulp(ref[0], "bf16"))
    assert np.abs(lse - ref[1]).max() <= 1e-3


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_extreme_scales_and_zero_blocks(kernel):
    """All value scales at either end of the supported range, or zero."""
    for s in (2.0 ** -60, 2.0 ** 60, 0.0):
        c = Case([1, 40, 300], 8, 16, "bf16", "e4m3", 16, seed=6)
        c.v_scales[:] = s
        ref = c.expected()
        o, lse = c.run(c.plan(flags=KERNELS[kernel], num_sms=3, ctas_per_sm=1,
                              min_chunk_tokens=16))
        if s == 0.0:
            assert np.all(o == 0)
        else:
            assert np.all(np.abs(o - ref[0]) <= 2e-3 * np.abs(ref[0]).max()
                          + np.abs(ref[0]) * 2.0 ** -8)
        assert np.abs(lse - ref[1]).max() <= 1e-3


def test_steep_and_negative_slopes():
    """Bias far beyond the scores: the nearest (or, negative, the first) token
    alone; zero slopes among them."""
    for group in (4, 8):
        c = Case([1000, 2, 513], group, 16, "f16", seed=8)
        n = 2 * group
        c.slopes = torch.tensor([[100.0, 0.0, -100.0, 1e-3][i % 4] for i in range(n)])
        ref = c.expected(alibi_slopes=c.slopes)
        for kw in SPLITS:
            got = c.run(c.plan(**kw), 0.0, True)
            assert_close(got[0], got[1] / np.maximum(1, np.abs(ref[1]) / 10), ref[0],
                         ref[1] / np.maximum(1, np.abs(ref[1]) / 10), "f16", str(kw))


@pytest.mark.parametrize("fmt", [None, "e4m3", "e5m2"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_options_with_rotary_positions(group, fmt):
    c = Case([1, 33, 700], group, 16, "bf16", fmt, 4 if fmt else 0, seed=9)
    ref = c.expected(logit_cap=20.0, alibi_slopes=c.slopes, rope_theta=1e4)
    for kw in SPLITS:
        _close(c.run(c.plan(rope_theta=1e4, **kw), 20.0, True), ref, "bf16", f"rope {fmt} {kw}")


def test_power_of_two_scales_equal_a_16bit_cache():
    """A 16-bit cache holding the same values: same result to rounding."""
    c = Case([300, 41], 4, 16, "bf16", "e4m3", 8, seed=10)
    for s in (c.k_scales, c.v_scales):
        s.copy_(torch.exp2(torch.round(torch.log2(s))))
    w = c.w
    ref = c.expected()
    got = c.run(c.plan())
    _close(got, ref, "bf16", "8-bit")
    from serving_attention_paged_b200.wrapper import PagedDecode
    pools = [torch.from_numpy(cache.cached_rows(p, np.arange(w.num_pages * 16), dtype="bf16",
                                                fmt="e4m3", scales=s, scale_block=8))
             .bfloat16().view(w.num_pages, 16, 2, 128).cuda()
             for p, s in zip(c.pools, (c.k_scales, c.v_scales))]
    pd = PagedDecode(w.kv_indptr, w.last_page_len, num_qo_heads=8, num_kv_heads=2, page_size=16,
                     dtype="bf16", sm_scale=w.sm_scale, num_pages=w.num_pages)
    o, lse = pd.run(c.q.cuda(), *pools, torch.from_numpy(w.kv_indices).cuda())
    _close((to_np(o), to_np(lse)), ref, "bf16", "16-bit")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
def test_prefill_cap_and_bias(group, dtype, causal):
    c = Case([200, 77, 1, 150, 64, 700], group, 16, dtype, seed=12, qo=[200, 40, 1, 0, 33, 300])
    from serving_attention_paged_b200.wrapper import PagedPrefill
    w = c.w
    for num_sms in (None, 2):
        pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=w.num_qo_heads,
                          num_kv_heads=w.num_kv_heads, page_size=16, dtype=dtype,
                          sm_scale=w.sm_scale, num_pages=w.num_pages, causal=causal,
                          num_sms=num_sms)
        # caps far below, near and far above the scores; with the mask also biased
        for cap, slopes in ((0.5, False), (5.0, causal), (50.0, causal), (0.0, causal)):
            if not cap and not slopes:
                continue
            got = c.run(pf, cap, slopes)
            ref = c.expected(qo_indptr=w.qo_indptr, causal=causal, logit_cap=cap,
                             alibi_slopes=c.slopes if slopes else None)
            assert_close(*got, *ref, dtype, f"cap={cap} {slopes} sms={num_sms}")


def test_prefill_sharp_scores_with_steep_bias():
    """Scores spread over tens of units under a bias that moves the maximum
    from tile to tile, and stale NaN rows behind the last key."""
    for dtype in ("f16", "bf16"):
        c = Case([1000, 300], 4, 16, dtype, seed=13, qo=[600, 300])
        w = c.w
        w.sm_scale = 1.0
        used = np.concatenate([cache._rows(b, w.kv_indptr, w.kv_indices, w.last_page_len, 16)
                               for b in range(2)])
        stale = np.setdiff1d(np.arange(w.num_pages * 16), used)
        for p in c.pools:
            p.view(-1, 2, 128)[torch.from_numpy(stale)] = float("nan")
        c.slopes = torch.tensor([3.0, 0.5, 0.05, 0.0] * 2)
        from serving_attention_paged_b200.wrapper import PagedPrefill
        pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=8,
                          num_kv_heads=2, page_size=16, dtype=dtype, sm_scale=1.0,
                          num_pages=w.num_pages)
        for cap in (0.0, 15.0):
            got = c.run(pf, cap, True)
            ref = c.expected(qo_indptr=w.qo_indptr, logit_cap=cap, alibi_slopes=c.slopes)
            # Where one or two tokens carry a row, fp16 P's rounding (half a
            # step, 2^-11 of each weight, the weights summing to 1 before it)
            # reaches o whole: |d o| <= sum 2^-11 p |v| <= 2^-11 max |v|.  The
            # exponentials on the FMA pipe add 7.5e-5 max |v|, the output its
            # half step.  max |v| is about 4.5 here, so 2e-3 alone is less than
            # that sum.  bf16 P keeps 16 bits.
            if dtype == "f16":
                vmax = np.abs(cache._widen16(c.pools[1].view(-1, 2, 128)[torch.from_numpy(used)],
                                             dtype)).max()
                allowed = (2.0 ** -11 + 7.5e-5) * vmax + half_ulp(ref[0], dtype) + 1e-4
                assert np.all(np.abs(got[0] - ref[0]) <= allowed), f"{dtype} cap={cap}"
                assert np.abs(got[1] - ref[1]).max() <= 1e-3
            else:
                assert_close(*got, *ref, dtype, f"{dtype} cap={cap}")


def test_append_decode_read_and_prefill_together():
    """A served sequence: prompts quantised as they are written, attended by
    unpacking into pages for the prefill, then tokens appended one by one and
    decoded over the codes, with the model's cap and bias."""
    from serving_attention_paged_b200.wrapper import PagedDecode, PagedKV, PagedPrefill
    P, hkv, hq, dtype, fmt, steps = 16, 2, 8, "bf16", "e4m3", 5
    prompts = [45, 16, 3]
    total = [n + steps for n in prompts]
    g = torch.Generator().manual_seed(1)
    x = {b: torch.randn(2, total[b], hkv, 128, generator=g).bfloat16() for b in range(3)}
    npages = sum(-(-n // P) for n in total) + 2
    order = np.random.default_rng(2).permutation(npages)
    start = np.concatenate([[0], np.cumsum([-(-n // P) for n in total])])
    codes = torch.zeros(2, npages, P, hkv, 128, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, npages, hkv, device="cuda")
    slopes = torch.exp2(-torch.arange(1, hq + 1).float())
    scale = 128 ** -0.5
    heads = dict(num_kv_heads=hkv, page_size=P, dtype=dtype, num_pages=npages)
    options = dict(logit_cap=30.0, alibi_slopes=slopes.cuda())
    ref_codes = [np.zeros((npages, P, hkv, 128), np.uint8) for _ in range(2)]
    ref_scales = [np.zeros((npages, hkv)) for _ in range(2)]

    def tables(lens):
        n = [-(-k // P) for k in lens]
        indptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        idx = np.concatenate([order[start[b]:start[b] + n[b]] for b in range(3)]).astype(np.int32)
        return indptr, idx, np.array([k - P * (m - 1) for k, m in zip(lens, n)], np.int32)

    def write(lens, new):
        indptr, idx, last = tables(lens)
        qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = torch.cat([x[b][:, lens[b] - new[b]:lens[b]] for b in range(3)], 1)
        pk = PagedKV(qo, indptr, last, kv_dtype=fmt, **heads)
        idx_d = torch.from_numpy(idx).cuda()
        pk.append(rows[0].cuda(), rows[1].cuda(), codes[0], codes[1], scales[0], scales[1], idx_d)
        for i in range(2):
            ref_codes[i], ref_scales[i] = cache.kv_append(
                rows[i], ref_codes[i], ref_scales[i], qo, indptr, idx, last, page_size=P,
                scale_block=P, dtype=dtype, fmt=fmt)
        return qo, indptr, idx, last, idx_d

    def expected(q, indptr, idx, last, qo=None):
        return cache.attention(q, ref_codes[0], ref_codes[1], indptr, idx, last, num_qo_heads=hq,
                               num_kv_heads=hkv, page_size=P, dtype=dtype, sm_scale=scale,
                               qo_indptr=qo, fmt=fmt, k_scales=ref_scales[0],
                               v_scales=ref_scales[1], scale_block=P, logit_cap=30.0,
                               alibi_slopes=slopes)

    qo, indptr, idx, last, idx_d = write(prompts, prompts)
    q = torch.randn(int(qo[-1]), hq, 128, generator=g).bfloat16()
    k16, v16 = (torch.zeros(len(idx), P, hkv, 128, dtype=torch.bfloat16, device="cuda")
                for _ in range(2))
    pages = torch.arange(len(idx), dtype=torch.int32, device="cuda")
    PagedKV(qo, indptr, last, kv_dtype=fmt, **heads).read(
        codes[0], codes[1], scales[0], scales[1], idx_d, k=k16, v=v16, out_indices=pages)
    pf = PagedPrefill(qo, indptr, last, num_qo_heads=hq, sm_scale=scale,
                      **{**heads, "num_pages": len(idx)})
    o, lse = pf.run(q.cuda(), k16, v16, pages, **options)
    assert_close(to_np(o), to_np(lse), *expected(q, indptr, idx, last, qo), dtype, "prefill")
    for step in range(1, steps + 1):
        lens = [n + step for n in prompts]
        _, indptr, idx, last, idx_d = write(lens, [1, 1, 1])
        q = torch.randn(3, hq, 128, generator=g).bfloat16()
        for flags in (0, 2):
            pd = PagedDecode(indptr, last, num_qo_heads=hq, sm_scale=scale, kv_dtype=fmt,
                             flags=flags, **heads)
            o, lse = pd.run(q.cuda(), codes[0], codes[1], idx_d, k_scales=scales[0],
                            v_scales=scales[1], **options)
            assert_close(to_np(o), to_np(lse), *expected(q, indptr, idx, last), dtype, str(step))


def test_captured_run_follows_new_scales_and_slopes():
    for flags in (2, 4):
        c = Case([300, 41, 0], 4, 16, "f16", "e4m3", 8, seed=14)
        pd = c.plan(flags=flags, num_sms=3, ctas_per_sm=1, min_chunk_tokens=32)
        dev = [c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(c.w.kv_indices).cuda()]
        ks, vs, sl = c.k_scales.cuda(), c.v_scales.cuda(), c.slopes.cuda()
        kw = dict(k_scales=ks, v_scales=vs, scale_block=8, logit_cap=25.0, alibi_slopes=sl)
        o, lse = pd.run(*dev, **kw)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            pd.run(*dev, o=o, lse=lse, **kw)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pd.run(*dev, o=o, lse=lse, **kw)
        for _ in range(2):
            for t, d in ((c.k_scales, ks), (c.v_scales, vs), (c.slopes, sl)):
                t *= 0.75
                d.copy_(t)
            g.replay()
            torch.cuda.synchronize()
            _close((to_np(o), to_np(lse)), c.expected(logit_cap=25.0, alibi_slopes=c.slopes),
                   "f16", "replay")


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_bad_page_is_reported_with_options(kernel):
    """Tokens of a bad page read as zeros, keys and values, as without options."""
    from serving_attention_paged_b200 import pagedattn as C
    c = Case([100, 70], 4, 16, "bf16", "e4m3", 16, seed=15)
    pd = c.plan(flags=KERNELS[kernel] | C.PA_FLAG_CHECK_INDICES)
    idx = c.w.kv_indices.copy()
    idx[2] = c.w.num_pages + 7
    o, lse = pd.run(c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(idx).cuda(),
                    k_scales=c.k_scales.cuda(), v_scales=c.v_scales.cuda(), scale_block=16)
    with pytest.raises(C.PagedAttnError) as e:
        pd.check()
    assert e.value.status == C.PA_ERR_DEVICE_CHECK and e.value.position == 2
    page = int(c.w.kv_indices[2])
    c.pools[0][page], c.pools[1][page] = 0, 0
    _close((to_np(o), to_np(lse)), c.expected(), "bf16", kernel)


def test_wrapper_refusals():
    from serving_attention_paged_b200 import pagedattn as C
    c = Case([40, 17], 4, 16, "f16", "e4m3", 8, seed=11)
    pd = c.plan()
    dev = [c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(c.w.kv_indices).cuda()]
    ks, vs, sl = c.k_scales.cuda(), c.v_scales.cuda(), c.slopes.cuda()
    for kw in (dict(k_scales=ks), dict(v_scales=vs), dict(scale_block=8),
               dict(k_scales=ks, v_scales=vs, scale_block=5),
               dict(k_scales=ks, v_scales=vs, scale_block=16),
               dict(k_scales=ks, v_scales=vs),                   # default: a page
               dict(k_scales=ks.half(), v_scales=vs, scale_block=8),
               dict(k_scales=ks.cpu(), v_scales=vs, scale_block=8),
               dict(alibi_slopes=sl[:-1]), dict(alibi_slopes=sl.double()),
               dict(alibi_slopes=sl.cpu())):
        with pytest.raises(ValueError):
            pd.run(*dev, **kw)
    for cap in (-1.0, float("nan"), float("inf"), 1e9, 1e-9):
        with pytest.raises(C.PagedAttnError):
            pd.run(*dev, logit_cap=cap)


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_cap_over_one_scale_per_tensor(kernel):
    """8-bit pools without block scales keep k_scale and v_scale."""
    from serving_attention_paged_b200.wrapper import PagedDecode
    w = W.make_workload("options", EDGE_LENS, num_qo_heads=8, num_kv_heads=2, page_size=16,
                        dtype="bf16", seed=21, kv_dtype="e5m2", k_scale=0.37, v_scale=1.3)
    t = w.materialize()
    slopes = torch.exp2(-torch.arange(1, 9).float())
    pd = PagedDecode(w.kv_indptr, w.last_page_len, num_qo_heads=8, num_kv_heads=2, page_size=16,
                     dtype="bf16", sm_scale=w.sm_scale, num_pages=w.num_pages, kv_dtype="e5m2",
                     k_scale=0.37, v_scale=1.3, flags=KERNELS[kernel], num_sms=3, ctas_per_sm=1,
                     min_chunk_tokens=64)
    o, lse = pd.run(t["q"].cuda(), t["k_pool"].cuda(), t["v_pool"].cuda(),
                    t["kv_indices"].cuda(), logit_cap=4.0, alibi_slopes=slopes.cuda())
    ref = cache.attention(t["q"], t["k_pool"], t["v_pool"], w.kv_indptr, w.kv_indices,
                          w.last_page_len, num_qo_heads=8, num_kv_heads=2, page_size=16,
                          dtype="bf16", sm_scale=w.sm_scale, fmt="e5m2", k_scale=0.37,
                          v_scale=1.3, logit_cap=4.0, alibi_slopes=slopes)
    assert_close(to_np(o), to_np(lse), *ref, "bf16", kernel)


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_negative_scales(kernel):
    c = Case([300, 5], 4, 16, "bf16", "e4m3", 4, seed=22)
    for s in (c.k_scales, c.v_scales):
        s[::3] *= -1
    _close(c.run(c.plan(flags=KERNELS[kernel])), c.expected(), "bf16", kernel)


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_many_small_weights_behind_a_sink(kernel):
    """One token takes nine tenths of the weight, 30,000 share the rest: each
    is 2^-18 of the largest, and together they move o by a tenth of V."""
    P, L = 64, 30000
    c = Case([L], 8, P, "bf16", "e4m3", P, hkv=1, seed=23, spread=0.0)
    w = c.w
    rows = cache._rows(0, w.kv_indptr, w.kv_indices, w.last_page_len, P)
    # every key 0 but the first, whose score is ln(9 (L - 1)) on every head
    c.pools[0].zero_()
    q = cache._widen16(c.q, "bf16").reshape(8, 128)
    key = np.linalg.pinv(q) @ np.full(8, np.log(9.0 * (L - 1)) / w.sm_scale)
    c.k_scales[:] = 2.0 ** -4
    c.pools[0].view(-1, 128)[int(rows[0])] = torch.from_numpy(cache.fp8_encode(key * 16, "e4m3"))
    # values: the sink's 0, the others' all 1 (code 64 * scale 1/64)
    c.v_scales[:] = 2.0 ** -6
    c.pools[1][:] = int(cache.fp8_encode([64.0], "e4m3")[0])
    c.pools[1].view(-1, 128)[int(rows[0])] = 0
    ref = c.expected()
    assert 0.02 < ref[0].mean() < 0.3
    for kw in SPLITS:
        o, lse = c.run(c.plan(flags=KERNELS[kernel], **kw))
        # each weight is kept to half of 2^-21 of the largest one, 2^-4 of itself, and a rounding
        # common to all equal weights; o is their mean: 2^-4 of 0.1 at most
        assert np.abs(o - ref[0]).max() <= 2.0 ** -4 * ref[0].max() + 2.0 ** -9
        assert np.abs(lse - ref[1]).max() <= 1e-3


def test_prefill_after_masked_tiles_and_odd_lengths():
    """New tokens around the 128-key tiles and the halves' bounds, so that a
    half's rows see no key of the item's last tile, for every group."""
    from serving_attention_paged_b200.wrapper import PagedPrefill
    for group, qo in ((1, [129, 257, 128, 300]), (2, [65, 129, 1, 130]), (8, [17, 33, 31, 16])):
        kv = [n + d for n, d in zip(qo, [0, 127, 128, 1])]
        c = Case(kv, group, 8, "bf16", seed=24, qo=qo)
        w = c.w
        pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=w.num_qo_heads,
                          num_kv_heads=2, page_size=8, dtype="bf16", sm_scale=w.sm_scale,
                          num_pages=w.num_pages, num_sms=3)
        for cap in (0.0, 3.0, 300.0):
            got = c.run(pf, cap, True)
            ref = c.expected(qo_indptr=w.qo_indptr, logit_cap=cap, alibi_slopes=c.slopes)
            assert_close(*got, *ref, "bf16", f"G={group} cap={cap}")


def test_options_on_another_stream():
    c = Case([300, 41], 4, 16, "f16", "e4m3", 8, seed=25)
    pd = c.plan()
    dev = [c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(c.w.kv_indices).cuda()]
    kw = dict(k_scales=c.k_scales.cuda(), v_scales=c.v_scales.cuda(), scale_block=8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = torch.empty(2, 8, 128, dtype=torch.float16, device="cuda"), torch.empty(2, 8, device="cuda")
    pd.run(*dev, o=o, lse=lse, stream=s, **kw)
    s.synchronize()
    ref = c.expected()
    _close((to_np(o), to_np(lse)), ref, "f16", "stream argument")
    with torch.cuda.stream(s):
        o2, lse2 = pd.run(*dev, **kw)
    s.synchronize()
    _close((to_np(o2), to_np(lse2)), ref, "f16", "current stream")


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_allocated_for_the_given_stream(handle):
    """Outputs that run makes for another stream (a Stream, or its handle) are
    no blocks on which the current stream's earlier work is still to come."""
    c = Case([300, 41], 4, 16, "f16", "e4m3", 8, seed=26)
    pd = c.plan()
    dev = [c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(c.w.kv_indices).cuda()]
    kw = dict(k_scales=c.k_scales.cuda(), v_scales=c.v_scales.cuda(), scale_block=8)
    want = pd.run(*dev, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(w) for w in want]
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for f in freed:
        f.fill_(7.0)
    del f, freed
    got = pd.run(*dev, stream=s.cuda_stream if handle else s, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
@pytest.mark.parametrize("fmt", [None, "e4m3"])
def test_distances_past_2_to_24(fmt, kernel):
    """A request of 2^24 + 37 tokens (one page of zeros repeated, then a last
    page of its own): keys 0, so the bias alone weighs, and the nearest
    distances must be exact integers.  o and lse in closed form."""
    from serving_attention_paged_b200.wrapper import PagedDecode
    P, hkv, G, last = 1024, 1, 4, 37
    n = (1 << 24) // P
    L = n * P + last
    indptr, indices = np.array([0, n + 1]), np.zeros(n + 1, np.int32)
    indices[-1] = 1
    slope = 0.25
    v = torch.zeros(2, P, hkv, 128)
    v[1, :last] = torch.randn(last, hkv, 128, generator=torch.Generator().manual_seed(4))
    k = torch.zeros(2, P, hkv, 128)
    kw = {}
    if fmt:
        v = torch.from_numpy(cache.fp8_encode(v.double().numpy() * 64, fmt))
        values = cache.fp8_table(fmt)[v.numpy()] / 64
        k = torch.zeros_like(v)
        kw = dict(k_scales=torch.ones(2, hkv, device="cuda"), scale_block=P,
                  v_scales=torch.full((2, hkv), 1 / 64, device="cuda"))
    else:
        k, v = k.bfloat16(), v.bfloat16()
        values = v.double().numpy()
    pd = PagedDecode(indptr, [last], num_qo_heads=hkv * G, num_kv_heads=hkv, page_size=P,
                     dtype="bf16", sm_scale=0.1, num_pages=2, kv_dtype=fmt, flags=KERNELS[kernel])
    q = torch.randn(1, hkv * G, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    o, lse = pd.run(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(indices).cuda(),
                    alibi_slopes=torch.full((G,), slope, device="cuda"), **kw)
    w = np.exp(-slope * np.arange(last)[::-1])       # of the last page's tokens
    z = (1 - np.exp(-slope * L)) / (1 - np.exp(-slope))
    ref = (w[:, None] * values[1, :last, 0]).sum(0) / z
    assert_close(to_np(o), to_np(lse), np.broadcast_to(ref, (1, G, 128)),
                 np.full((1, G), np.log(z)), "bf16", kernel)


def test_prefill_options_report_a_bad_page():
    from serving_attention_paged_b200 import pagedattn as C
    from serving_attention_paged_b200.wrapper import PagedPrefill
    c = Case([100, 70], 4, 16, "bf16", seed=26, qo=[100, 20])
    w = c.w
    pf = PagedPrefill(w.qo_indptr, w.kv_indptr, w.last_page_len, num_qo_heads=8, num_kv_heads=2,
                      page_size=16, dtype="bf16", sm_scale=w.sm_scale, num_pages=w.num_pages,
                      flags=C.PA_FLAG_CHECK_INDICES)
    idx = w.kv_indices.copy()
    idx[3] = -2
    o, lse = pf.run(c.q.cuda(), *[p.cuda() for p in c.pools], torch.from_numpy(idx).cuda(),
                    logit_cap=10.0, alibi_slopes=c.slopes.cuda())
    with pytest.raises(C.PagedAttnError) as e:
        pf.check()
    assert e.value.position == 3
    page = int(w.kv_indices[3])
    c.pools[0][page], c.pools[1][page] = 0, 0  # its tokens read as zeros
    ref = c.expected(qo_indptr=w.qo_indptr, logit_cap=10.0, alibi_slopes=c.slopes)
    assert_close(to_np(o), to_np(lse), *ref, "bf16", "bad page")
