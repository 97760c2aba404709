"""Writing and reading the block-scaled 8-bit KV cache on the GPU, against the
fp64 definition in oracle/cache.py.

Every step of the quantisation is exact but the rounding of the code itself
(scales are powers of two, so quotients are exact in fp32): codes and scales
are compared bit for bit, over the whole pools, so that what must not be
touched is checked too.  Reading back is scale * code rounded once.
"""
import numpy as np
import pytest
import torch

from oracle import cache
from serving_attention_paged_b200 import workloads as W

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {"f16": torch.float16, "bf16": torch.bfloat16}


class Cache:
    """Random pools and scales (stale contents), tables and new rows."""

    def __init__(self, lens, new, P, block, dtype, fmt, hkv=2, seed=0, extra=3, pow2=True):
        self.P, self.block, self.dtype, self.fmt, self.hkv = P, block, dtype, fmt, hkv
        self.lens, self.new = lens, new
        g = torch.Generator().manual_seed(seed)
        n = sum(-(-x // P) for x in lens) + extra
        self.indptr, self.indices, self.last = W.tables_from_lengths(
            lens, P, np.random.default_rng(seed).permutation(n))
        self.num_pages = n
        self.qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        finite = np.nonzero(np.isfinite(cache.fp8_table(fmt)))[0].astype(np.uint8)
        shape = (n, P, hkv, 128)
        self.codes = [torch.from_numpy(finite)[torch.randint(len(finite), shape, generator=g)]
                      for _ in range(2)]
        s = torch.randint(-8, 3, (2, n * P // block, hkv), generator=g)
        self.scales = torch.exp2(s.float())
        if not pow2:
            self.scales *= 1 + torch.rand(self.scales.shape, generator=g)
        mag = torch.exp2(torch.randint(-6, 7, (2, int(self.qo[-1]), hkv, 1), generator=g).float())
        self.x = (torch.randn(2, int(self.qo[-1]), hkv, 128, generator=g) * mag).to(HALF[dtype])

    def expected(self, which):
        return cache.kv_append(self.x[which], self.codes[which].numpy(),
                               self.scales[which].numpy(), self.qo, self.indptr, self.indices,
                               self.last, page_size=self.P, scale_block=self.block,
                               dtype=self.dtype, fmt=self.fmt)

    def plan(self, qo=None, **kw):
        from serving_attention_paged_b200.wrapper import PagedKV
        return PagedKV(self.qo if qo is None else qo, self.indptr, self.last,
                       num_kv_heads=self.hkv, page_size=self.P, dtype=self.dtype,
                       kv_dtype=self.fmt, num_pages=self.num_pages, scale_block=self.block, **kw)

    def device(self):
        pools = [c.cuda() for c in self.codes]
        scales = [s.clone().cuda() for s in self.scales]
        return (*pools, *scales, torch.from_numpy(self.indices).cuda())


def _check_append(c, dev, what=""):
    for w in range(2):
        codes, scales = c.expected(w)
        assert np.array_equal(dev[2 + w].cpu().numpy().astype(np.float64), scales), what
        assert np.array_equal(dev[w].cpu().numpy(), codes), what


LENS = [37, 0, 1, 16, 90, 33, 64, 200, 5]
NEW = {"one": [1, 0, 1, 1, 1, 1, 1, 1, 1], "all": LENS, "some": [20, 0, 0, 16, 45, 2, 17, 133, 3]}
PAGES = [(1, 1), (2, 2), (8, 4), (8, 8), (16, 1), (16, 2), (16, 16), (64, 8), (32, 32), (64, 64),
         (128, 16), (256, 128), (1024, 256), (1024, 1024)]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("P,block", PAGES)
def test_append_bitwise(P, block, dtype, fmt):
    for k, (name, new) in enumerate(NEW.items()):
        lens = [n * (P // 64) + 1 if P > 128 and n else n for n in LENS]
        new = lens if name == "all" else new
        c = Cache(lens, new, P, block, dtype, fmt, hkv=[1, 2, 3][k], seed=P + block + k)
        dev = c.device()
        pk = c.plan()
        x = c.x.cuda()
        pk.append(x[0], x[1], *dev)
        assert pk.check() == -1
        _check_append(c, dev, f"{name} P={P} block={block}")
        pk.append(x[0], x[1], *dev)  # again: the scales no longer grow
        _check_append(c, dev, "again")


def test_append_special_values():
    """Zeros, subnormals, infinities and NaN among the rows: a block without a
    finite value or of zeros gets the smallest scale, non-finite elements
    leave the others' scale alone."""
    for dtype in ("f16", "bf16"):
        for block in (1, 16, 64):
            c = Cache([64, 130], [40, 129], 64, block, dtype, "e4m3", seed=block)
            x = c.x
            x[:, 0] = 0
            x[:, 1, :, ::3] = float("inf")
            x[:, 2, :, 1::2] = float("nan")
            x[:, 3] = float("nan")
            x[:, 4] = -float("inf")
            x[:, 5] = torch.finfo(x.dtype).tiny / 4
            x[:, 6] = torch.finfo(x.dtype).max
            x[:, 60:, :, 5] = 0.0
            x[:, 60:, :, 6] = -0.0
            dev = c.device()
            c.plan().append(x[0].cuda(), x[1].cuda(), *dev)
            _check_append(c, dev, f"{dtype} {block}")


def test_append_from_strided_rows_and_head_counts():
    """K and V as slices of one projection's rows, at different strides."""
    for hkv in (1, 5, 8):
        c = Cache([50, 33, 16], [50, 12, 1], 16, 16, "bf16", "e4m3", hkv=hkv, seed=hkv)
        wide = torch.zeros(int(c.qo[-1]), 4 + 2 * hkv, 128, dtype=torch.bfloat16)
        wide[:, 2:2 + hkv], wide[:, -hkv:] = c.x[0], c.x[1]
        wide = wide.cuda()
        dev = c.device()
        c.plan().append(wide[:, 2:2 + hkv], wide[:, -hkv:], *dev)
        _check_append(c, dev)


@pytest.mark.parametrize("block", [4, 64])
def test_append_into_blocks_with_other_scales(block):
    """Earlier scales that are no powers of two (another writer's): kept where
    large enough, codes within half a step of x / scale (one fp32 rounding of
    the quotient on top: 2^-23 relative covers it)."""
    c = Cache([37, 90, 130], [1, 3, 40], 64, block, "f16", "e4m3", seed=9, pow2=False)
    dev = c.device()
    c.plan().append(c.x[0].cuda(), c.x[1].cuda(), *dev)
    table = cache.fp8_table("e4m3")
    for w in range(2):
        codes, scales = c.expected(w)
        # scales: old, or a power of two; both exact
        assert np.array_equal(dev[2 + w].cpu().numpy().astype(np.float64), scales)
        for b in range(3):
            rows = cache._rows(b, c.indptr, c.indices, c.last, 64)[c.lens[b] - c.new[b]:]
            got = table[dev[w].cpu().numpy().reshape(-1, 2, 128)[rows]]
            s = scales.reshape(-1, 2)[rows // block][..., None]
            y = c.x[w][c.qo[b]:c.qo[b + 1]].double().numpy() / s
            # half a step: 2^-4 relative, or half of the smallest subnormal 2^-9
            assert np.all(np.abs(got - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10)
                          * (1 + 2.0 ** -22))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("P,block", PAGES)
def test_read_rows(P, block, dtype, fmt):
    for name, new in NEW.items():
        c = Cache(LENS, new, P, block, dtype, fmt, seed=2 * P + block)
        dev = c.device()
        guard = torch.full((int(c.qo[-1]) + 2, c.hkv + 1, 128), 7.0, dtype=HALF[dtype],
                           device="cuda")
        k, v = guard[1:-1, :c.hkv], torch.empty(int(c.qo[-1]), c.hkv, 128, dtype=HALF[dtype],
                                                device="cuda")
        pk = c.plan()
        pk.read(*dev, k=k, v=v)
        assert pk.check() == -1
        for w, got in enumerate((k, v)):
            ref = cache.kv_read(c.codes[w].numpy(), c.scales[w], c.indptr, c.indices, c.last,
                                page_size=P, scale_block=block, dtype=dtype, fmt=fmt, new=new)
            # powers of two: the product is exact, one rounding remains
            assert torch.equal(got.cpu(), torch.from_numpy(ref).to(HALF[dtype])), name
        assert (guard[0] == 7).all() and (guard[-1] == 7).all() and (guard[:, c.hkv:] == 7).all()


def test_read_with_any_scales_rounds_once():
    c = Cache([300, 17], [300, 9], 16, 4, "bf16", "e5m2", seed=4, pow2=False)
    dev = c.device()
    k, v = c.plan().read(*dev)
    for w, got in enumerate((k, v)):
        ref = cache.kv_read(c.codes[w].numpy(), c.scales[w], c.indptr, c.indices, c.last,
                            page_size=16, scale_block=4, dtype="bf16", fmt="e5m2", new=c.new)
        err = np.abs(got.double().cpu().numpy() - ref)
        # half a bf16 step, plus the fp32 product's own rounding
        assert np.all(err <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -24))


@pytest.mark.parametrize("P,block", [(8, 2), (16, 16), (64, 64), (1024, 256)])
def test_read_into_pages(P, block):
    """Into pages of a 16-bit pool chosen by out_indices; other rows keep
    their contents, rows of a last page past its tokens included."""
    c = Cache(LENS, LENS, P, block, "f16", "e4m3", seed=P)
    dev = c.device()
    n_out = c.num_pages + 5
    out = np.random.default_rng(1).permutation(n_out)[:len(c.indices)].astype(np.int32)
    pools = [torch.full((n_out, P, c.hkv, 128), 3.0, dtype=torch.float16, device="cuda")
             for _ in range(2)]
    pk = c.plan(flags=1)
    pk.read(*dev, k=pools[0], v=pools[1], out_indices=torch.from_numpy(out).cuda())
    assert pk.check() == -1
    for w in range(2):
        ref = torch.full((n_out * P, c.hkv, 128), 3.0, dtype=torch.float16)
        for b in range(len(LENS)):
            src = cache._rows(b, c.indptr, c.indices, c.last, P)
            dst = cache._rows(b, c.indptr, out, c.last, P)
            x = cache.cached_rows(c.codes[w].numpy(), src, dtype="f16", fmt="e4m3",
                                  scales=c.scales[w], scale_block=block)
            ref[torch.from_numpy(dst)] = torch.from_numpy(x).half()
        assert torch.equal(pools[w].cpu().view(-1, c.hkv, 128), ref)


@pytest.mark.parametrize("block", [4, 16, 64])
def test_bad_pages_are_skipped_and_reported(block):
    from serving_attention_paged_b200 import pagedattn as C
    c = Cache([100, 70], [90, 70], 64, block, "bf16", "e4m3", seed=8)
    dev = c.device()
    bad = c.indices.copy()
    bad[1] = c.num_pages      # request 0, tokens 64 .. 99
    bad[3] = -1               # request 1, tokens 64 .. 69
    pk = c.plan(flags=C.PA_FLAG_CHECK_INDICES)
    pk.append(c.x[0].cuda(), c.x[1].cuda(), *dev[:4], torch.from_numpy(bad).cuda())
    with pytest.raises(C.PagedAttnError) as e:
        pk.check()
    assert e.value.position == 1
    assert pk.check() == -1  # cleared
    for w in range(2):
        codes, scales = c.expected(w)
        keep = torch.from_numpy(c.indices[[1, 3]].astype(np.int64))
        codes[keep] = c.codes[w][keep].numpy()  # as before on the two pages' places
        per = 64 // block
        scales = scales.reshape(-1, per, c.hkv)
        scales[keep] = c.scales[w].view(-1, per, c.hkv)[keep].double().numpy()
        assert np.array_equal(dev[w].cpu().numpy(), codes)
        assert np.array_equal(dev[2 + w].cpu().numpy().astype(np.float64).reshape(scales.shape),
                              scales)
    k = torch.full((160, c.hkv, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    pk.read(*dev[:4], torch.from_numpy(bad).cuda(), k=k, v=v)
    with pytest.raises(C.PagedAttnError) as e:
        pk.check()
    assert e.value.position == 1
    # request 0's new tokens are 10 .. 99: rows 54 .. 89 lie on the bad page
    assert (k[54:90] == 5).all() and (v[154:] == 5).all() and not (k[:54] == 5).all()


def test_captured_append_and_read_replay_on_new_rows():
    c = Cache([40, 17], [8, 17], 16, 8, "f16", "e4m3", seed=11)
    dev = c.device()
    x = c.x.cuda()
    pk = c.plan()
    other = c.plan()  # two plans' workspaces in one graph
    k, v = pk.read(*dev)
    start = [d.clone() for d in dev]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pk.append(x[0], x[1], *dev)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.append(x[0], x[1], *dev)
        other.read(*dev, k=k, v=v)
    for seed in (12, 13):
        c2 = Cache([40, 17], [8, 17], 16, 8, "f16", "e4m3", seed=seed)
        c.x = c2.x
        x.copy_(c2.x)
        for d, st in zip(dev, start):
            d.copy_(st)
        g.replay()
        torch.cuda.synchronize()
        _check_append(c, dev)
        codes, scales = c.expected(0)
        ref = cache.kv_read(codes, scales, c.indptr, c.indices, c.last, page_size=16,
                            scale_block=8, dtype="f16", fmt="e4m3", new=c.new)
        assert torch.equal(k.cpu(), torch.from_numpy(ref).half())


def test_wrapper_refusals():
    c = Cache([40, 17], [8, 17], 16, 8, "f16", "e4m3", seed=11)
    dev = c.device()
    x = c.x.cuda()
    pk = c.plan()

    def refused(call):
        with pytest.raises(ValueError):
            call()

    refused(lambda: pk.append(x[0].bfloat16(), x[1], *dev))
    refused(lambda: pk.append(x[0, :-1], x[1], *dev))
    refused(lambda: pk.append(x[0].cpu(), x[1], *dev))
    refused(lambda: pk.append(x[0].transpose(1, 2).contiguous().transpose(1, 2), x[1], *dev))
    refused(lambda: pk.append(x[0], x[1], dev[0][:-1], *dev[1:]))
    refused(lambda: pk.append(x[0], x[1], dev[0].view(torch.float8_e5m2), *dev[1:]))
    refused(lambda: pk.append(x[0], x[1], *dev[:2], dev[2].half(), *dev[3:]))
    refused(lambda: pk.append(x[0], x[1], *dev[:2], dev[2][:-1], *dev[3:]))
    refused(lambda: pk.append(x[0], x[1], *dev[:4], dev[4].long()))
    refused(lambda: pk.append(x[0], x[1], *dev[:4], dev[4][:-1]))
    refused(lambda: pk.read(*dev, out_indices=dev[4]))
    refused(lambda: pk.read(*dev, k=x[0].float()))


def test_empty_plans_and_empty_batch():
    c = Cache([40, 0], [0, 0], 16, 8, "f16", "e4m3", seed=1)
    dev = c.device()
    before = [d.clone() for d in dev]
    pk = c.plan()
    pk.append(c.x[0].cuda(), c.x[1].cuda(), *dev)
    k, v = pk.read(*dev)
    assert k.shape == v.shape == (0, 2, 128)
    assert all(torch.equal(a, b) for a, b in zip(before, dev))
    from serving_attention_paged_b200.wrapper import PagedKV
    empty = PagedKV([0], [0], [], num_kv_heads=2, page_size=16, dtype="f16", kv_dtype="e4m3",
                    num_pages=c.num_pages, scale_block=8)
    empty.append(c.x[0].cuda(), c.x[1].cuda(), *dev)
    assert empty.check() == -1


def test_pool_offsets_past_32_bits():
    """Rows whose byte offset passes 2^32: the last pages of a 5 GB pool."""
    from serving_attention_paged_b200.wrapper import PagedDecode, PagedKV
    P, hkv, n = 64, 8, 80000                    # 80,000 x 64 x 1 KB = 5.2 GB per pool
    lens = [100, 33]
    indptr, _, last = W.tables_from_lengths(lens, P)
    idx = np.array([n - 1, n - 3, n - 2], dtype=np.int32)
    pools = [torch.empty(n, P, hkv, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(n, hkv, device="cuda") for _ in range(2)]
    before = [p[:4].clone() for p in pools]
    qo = np.array([0, 100, 133], dtype=np.int32)
    x = torch.randn(2, 133, hkv, 128, generator=torch.Generator().manual_seed(0)).bfloat16()
    pk = PagedKV(qo, indptr, last, num_kv_heads=hkv, page_size=P, dtype="bf16", kv_dtype="e4m3",
                 num_pages=n)
    idx_d = torch.from_numpy(idx).cuda()
    pk.append(x[0].cuda(), x[1].cuda(), *pools, *scales, idx_d)
    back = pk.read(*pools, *scales, idx_d)
    small = np.array([2, 0, 1], dtype=np.int32)  # the same pages, of a pool of three
    for w in range(2):
        codes, s = cache.kv_append(x[w], np.zeros((3, P, hkv, 128), np.uint8), np.ones((3, hkv)),
                                   qo, indptr, small, last, page_size=P, scale_block=P,
                                   dtype="bf16", fmt="e4m3")
        ref = cache.kv_read(codes, s, indptr, small, last, page_size=P, scale_block=P,
                            dtype="bf16", fmt="e4m3")
        assert torch.equal(back[w].cpu(), torch.from_numpy(ref).bfloat16())
        assert torch.equal(pools[w][:4], before[w])
    q = torch.randn(2, 32, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    args = [cache.kv_append(x[w], np.zeros((3, P, hkv, 128), np.uint8), np.ones((3, hkv)), qo,
                            indptr, small, last, page_size=P, scale_block=P, dtype="bf16",
                            fmt="e4m3") for w in range(2)]
    ref = cache.attention(q, args[0][0], args[1][0], indptr, small, last, num_qo_heads=32,
                          num_kv_heads=hkv, page_size=P, dtype="bf16", sm_scale=0.0884,
                          fmt="e4m3", k_scales=args[0][1], v_scales=args[1][1], scale_block=P)
    for flags in (2, 4):
        pd = PagedDecode(indptr, last, num_qo_heads=32, num_kv_heads=hkv, page_size=P,
                         dtype="bf16", sm_scale=0.0884, num_pages=n, kv_dtype="e4m3", flags=flags)
        o, lse = pd.run(q.cuda(), *pools, idx_d, k_scales=scales[0], v_scales=scales[1])
        assert np.abs(o.double().cpu().numpy() - ref[0]).max() <= 2e-3 + 2.0 ** -8 * 4.5
        assert np.abs(lse.double().cpu().numpy() - ref[1]).max() <= 1e-3


def test_two_plans_into_one_cache_and_a_given_stream():
    """Two appends of different requests into one pool, one after the other on
    another stream than the current one."""
    c = Cache([40, 17, 90], [40, 17, 90], 16, 16, "f16", "e4m3", seed=31)
    dev = c.device()
    x = c.x.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    from serving_attention_paged_b200.wrapper import PagedKV
    for b0, b1 in ((0, 1), (1, 3)):
        p0, p1 = int(c.indptr[b0]), int(c.indptr[b1])
        pk = PagedKV(c.qo[b0:b1 + 1] - c.qo[b0], c.indptr[b0:b1 + 1] - p0, c.last[b0:b1],
                     num_kv_heads=2, page_size=16, dtype="f16", kv_dtype="e4m3",
                     num_pages=c.num_pages, scale_block=16, stream=s)
        rows = slice(int(c.qo[b0]), int(c.qo[b1]))
        idx = torch.from_numpy(c.indices[p0:p1]).cuda()
        torch.cuda.synchronize()
        pk.append(x[0, rows], x[1, rows], *dev[:4], idx, stream=s)
        s.synchronize()
    _check_append(c, dev)


def test_negative_pages_are_skipped_without_the_check():
    c = Cache([40], [40], 16, 16, "f16", "e4m3", seed=41)
    dev = c.device()
    idx = c.indices.copy()
    idx[1] = -1
    c.plan().append(c.x[0].cuda(), c.x[1].cuda(), *dev[:4], torch.from_numpy(idx).cuda())
    for w in range(2):
        codes, scales = c.expected(w)
        page = int(c.indices[1])
        codes[page], scales[page] = c.codes[w][page].numpy(), c.scales[w][page].numpy()
        assert np.array_equal(dev[w].cpu().numpy(), codes)
        assert np.array_equal(dev[2 + w].cpu().numpy().astype(np.float64), scales)


def test_single_head_rows_at_any_inner_stride():
    """One kv head: the stride of the heads' axis says nothing."""
    c = Cache([40, 3], [40, 3], 16, 16, "bf16", "e4m3", hkv=1, seed=42)
    dev = c.device()
    x = [torch.empty_strided((43, 1, 128), (128, 7, 1), dtype=torch.bfloat16, device="cuda")
         for _ in range(2)]
    for a, b in zip(x, c.x):
        a.copy_(b)
    c.plan().append(*x, *dev)
    _check_append(c, dev)


def test_read_allocates_for_the_given_stream():
    """Outputs that read makes for another stream are no blocks on which the
    current stream's earlier work is still to come."""
    c = Cache([40, 17], [40, 17], 16, 16, "f16", "e4m3", seed=43)
    dev = c.device()
    pk = c.plan()
    pk.append(c.x[0].cuda(), c.x[1].cuda(), *dev)
    want = pk.read(*dev)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.empty_like(w) for w in want]
    torch.cuda._sleep(100_000_000)  # some 50 ms
    for f in freed:
        f.fill_(7.0)
    del f, freed
    got = pk.read(*dev, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("check", [False, True])
@pytest.mark.parametrize("block", [4, 16, 64])
def test_read_makes_zeros_of_bad_pages(block, check):
    """Rows that read makes itself hold nothing of the allocator's last user:
    tokens on a bad page are zeros, as attention takes them."""
    from serving_attention_paged_b200 import pagedattn as C
    c = Cache([100, 70], [90, 70], 64, block, "bf16", "e4m3", seed=50)
    dev = c.device()
    bad = c.indices.copy()
    bad[1] = c.num_pages if check else -5  # request 0, tokens 64 .. 99: rows 54 .. 89
    bad[3] = -1                            # request 1, tokens 64 .. 69: the last 6 rows
    pk = c.plan(flags=C.PA_FLAG_CHECK_INDICES if check else 0)
    good = pk.read(*dev)
    idx = torch.from_numpy(bad).cuda()

    def verify(got):
        want = torch.where(zero[:, None, None], torch.zeros((), dtype=torch.bfloat16), good[w].cpu())
        assert torch.equal(got.cpu(), want)

    zero = torch.zeros(160, dtype=torch.bool)
    zero[54:90], zero[154:] = True, True
    for given in (None, "k", "v"):
        torch.cuda.synchronize()
        dirty = [torch.full((160, c.hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
                 for _ in range(2)]
        del dirty  # the next blocks of this size
        mine = torch.full((160, c.hkv, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        got = pk.read(*dev[:4], idx, **({given: mine} if given else {}))
        torch.cuda.synchronize()
        for w, name in enumerate("kv"):
            if name == given:
                assert got[w] is mine and (mine[54:90] == 5).all() and (mine[154:] == 5).all()
                assert torch.equal(mine[:54], good[w][:54])
            else:
                verify(got[w])
    if check:
        with pytest.raises(C.PagedAttnError):
            pk.check()
