"""Attention with options where many tokens weigh little: one token (an
attention sink) takes nine tenths of the softmax, a long tail shares the rest.

Whatever resolution a kernel's weights have, what it keeps of the tail has to
add up: o stays within the library's 2e-3 at any length.  The references are
closed forms in 64 bits: the tail is one page, read again and again.
"""
import numpy as np
import pytest
import torch

from oracle import cache
from parity import assert_close, to_np

pytestmark = pytest.mark.gpu

P, D, G = 1024, 128, 8
KERNELS = {"cuda_cores": 2, "tensor_cores": 4}
HALF = {"f16": torch.float16, "bf16": torch.bfloat16}


class Tail:
    """n pages of tokens: the first page's first token is the sink, of score
    `top`; every other token t of a page scores top * c[t] and has value v[t],
    the same on each page.  The key is one element, c = 1 for the sink."""

    def __init__(self, pages, weight, spread, seed=0):
        g = np.random.default_rng(seed)
        self.top = -np.log(weight)  # the tail's c is around 0
        self.c = np.zeros(P)
        if spread:  # normal scores, so log-normal weights
            self.c = np.clip(g.normal(size=P) * spread / self.top, -0.4, 0.4)
            self.c = cache.fp8_table("e4m3")[cache.fp8_encode(self.c, "e4m3")]
        v = 1.0 + 0.25 * g.normal(size=(P, D))
        self.v = cache.fp8_table("e4m3")[cache.fp8_encode(v * 16, "e4m3")] / 16
        self.pages = pages

    def expected(self):
        """o [D], lse; the sink's value is 0."""
        w = np.exp(self.top * (self.c - 1.0))  # relative to the sink
        total = 1.0 + (self.pages - 1) * w.sum() + w[1:].sum()
        o = ((self.pages - 1) * w @ self.v + w[1:] @ self.v[1:]) / total
        return o, self.top + np.log(total)

    def pools(self):
        """[2 pages, P, 1, D] keys and values: the tail's page, the first page."""
        k, v = np.zeros((2, 2, P, 1, D))
        k[:, :, 0, 0] = self.c
        v[:, :, 0] = self.v
        k[1, 0, 0, 0], v[1, 0, 0] = 1.0, 0.0
        return k, v

    def tables(self):
        indices = np.zeros(self.pages, np.int32)
        indices[0] = 1
        return [0, self.pages], [P], indices


def _decode(case, dtype, kernel, fmt, **kw):
    """One unsplit piece, G heads with the same query."""
    from serving_attention_paged_b200.wrapper import PagedDecode
    indptr, last, indices = case.tables()
    pd = PagedDecode(indptr, last, num_qo_heads=G, num_kv_heads=1, page_size=P, dtype=dtype,
                     sm_scale=case.top, num_pages=2, kv_dtype=fmt, flags=KERNELS[kernel],
                     num_sms=1, ctas_per_sm=1)
    k, v = case.pools()
    if fmt:
        k, v = (torch.from_numpy(cache.fp8_encode(x * 16, fmt)) for x in (k, v))
        s = torch.full((2, 1), 1 / 16, device="cuda")
        kw.update(k_scales=s, v_scales=s, scale_block=P)
    else:
        k, v = (torch.from_numpy(x).to(HALF[dtype]) for x in (k, v))
    q = torch.zeros(1, G, D, dtype=HALF[dtype])
    q[..., 0] = 1.0
    o, lse = pd.run(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(indices).cuda(), **kw)
    torch.cuda.synchronize()
    assert pd.check() == -1
    return to_np(o), to_np(lse)


def _close(got, o, lse, dtype, what, lse_more=0.0):
    assert np.isfinite(got[0]).all(), what
    o = np.broadcast_to(o, got[0].shape)
    off = got[1] - lse
    assert_close(got[0], lse + np.sign(off) * np.maximum(np.abs(off) - lse_more, 0), o,
                 np.full(got[1].shape, lse), dtype, what)


# (pages, a token's weight relative to the sink's, spread of the tail's scores).
# The equal weights lie half way between two steps of 2^-21 and of 2^-25 of the
# largest weight; their sum is about a tenth of the whole.
TAILS = [(128, 1.5 * 2.0 ** -21, 0.0), (512, 2.0 ** -22, 1.0), (2048, 1.5 * 2.0 ** -25, 0.0),
         (2048, 2.0 ** -25, 1.5)]


@pytest.mark.parametrize("pages,weight,spread", TAILS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_tail_behind_a_sink_in_an_8bit_cache(kernel, dtype, pages, weight, spread):
    case = Tail(pages, weight, spread)
    o, lse = case.expected()
    assert 0.03 < o.mean() < 0.5
    got = _decode(case, dtype, kernel, "e4m3")
    # The thread that holds the sink adds a tile's share of the tail to a sum of
    # 1 or a little more, each time off by half an fp32 step of it, 2^-24: after
    # 2^21 tokens the lse may be off by that for each of its tiles (of 32 tokens
    # on the CUDA cores, of 256 on the tensor cores).
    sums = pages * P / (32 if kernel == "cuda_cores" else 256) * 2.0 ** -24
    _close(got, o, lse, dtype, kernel, sums)


@pytest.mark.parametrize("spread", [12, 16, 20])
@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_values_beside_a_block_of_far_larger_scale(kernel, spread):
    """4,096 tokens of log-normal weights, 1 on average; one block's tokens
    weigh 1 each, its V scale is 2^spread the others' and its codes are 0 in
    half of the elements.  There o is the others' alone.  A weight of the
    large block is 2^4 of the P V's units or more, the others' 2^(4 - spread)
    on average; what the tensor-core kernel drops of them stays below 2^-22
    for each of a tile's 256 places, so o is off by 256 * 2^-22 / (4,096 *
    2^(4 - spread)) = 2^(spread - 30) of itself: 2^-10 at most, below 2e-3."""
    from serving_attention_paged_b200.wrapper import PagedDecode
    page, n, block = 16, 4096, 37
    scores = np.random.default_rng(spread).normal(size=n // page * page) * 0.5
    k = np.zeros((n // page, page, 1, D))
    k[..., 0] = scores.reshape(n // page, page, 1)
    k[block] = 0.0
    codes = cache.fp8_encode(k, "e4m3")
    w = np.exp(cache.fp8_table("e4m3")[codes[..., 0]]).reshape(n // page, page)
    assert w.mean() > 1.0
    v = np.ones((n // page, page, 1, D))
    v[block, :, :, D // 2:] = 0.0
    vs = torch.ones(n // page, 1)
    vs[block] = 2.0 ** spread
    pd = PagedDecode([0, n // page], [page], num_qo_heads=G, num_kv_heads=1, page_size=page,
                     dtype="bf16", sm_scale=1.0, num_pages=n // page, kv_dtype="e4m3",
                     flags=KERNELS[kernel], num_sms=1, ctas_per_sm=1)
    q = torch.zeros(1, G, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    o, lse = pd.run(q.cuda(), torch.from_numpy(codes).cuda(),
                    torch.from_numpy(cache.fp8_encode(v, "e4m3")).cuda(),
                    torch.arange(n // page, dtype=torch.int32, device="cuda"),
                    k_scales=torch.ones(n // page, 1, device="cuda"), v_scales=vs.cuda())
    small = (w.sum() - page) / w.sum()
    large = small + page * 2.0 ** spread / w.sum()
    ref = np.concatenate([np.full(D // 2, large), np.full(D // 2, small)])
    # bf16 rounds the output by up to 2^-8 of it
    assert np.all(np.abs(to_np(o) - ref) <= (2e-3 + 2.0 ** -8) * ref)
    assert np.abs(to_np(lse) - np.log(w.sum())).max() <= 1e-3


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kernel", ["cuda_cores", "tensor_cores"])
def test_tail_behind_a_sink_in_a_16bit_cache(kernel, dtype):
    """Equal weights of 12.5 and 1.5 steps of 2^-24 of the largest: fp16's
    subnormals."""
    for pages, weight in ((128, 12.5 * 2.0 ** -24), (1024, 1.5 * 2.0 ** -24)):
        case = Tail(pages, weight, 0.0)
        o, lse = case.expected()
        got = _decode(case, dtype, kernel, None, alibi_slopes=torch.zeros(G, device="cuda"))
        sums = pages * P / (32 if kernel == "cuda_cores" else 128) * 2.0 ** -24
        _close(got, o, lse, dtype, kernel, sums)
