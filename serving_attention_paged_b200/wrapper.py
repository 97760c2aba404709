"""Convenience layer over the C ABI for PyTorch callers.

``PagedDecode`` holds a plan and its device workspace (allocated through
torch, the library itself never allocates) and calls ``pa_run`` /
``pa_cascade_run``; ``PagedPrefill`` does the same for ``pa_prefill_run`` and
``PagedKV`` for ``pa_kv_append`` / ``pa_kv_read`` (8-bit caches with a scale
for each block of tokens and kv head).  They only marshal arguments; all attention work is done by the library's
kernels.
"""
from __future__ import annotations

import torch

from . import pagedattn as C

_TORCH_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


_KV8_DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _device(device) -> torch.device:
    """The given device (default: the current one), with its index."""
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _require(ok, what):
    if not ok:
        raise ValueError(what)


def _check_scales(k_scales, v_scales, blocks, num_kv_heads, dev):
    n = blocks * num_kv_heads
    for x in (k_scales, v_scales):
        if not (x.dtype is torch.float32 and x.numel() == n and x.get_device() == dev
                and x.is_contiguous()):
            raise ValueError(f"k_scales and v_scales: contiguous float32 [{blocks}, "
                             f"{num_kv_heads}] (blocks of tokens of the pool, kv heads) on "
                             f"cuda:{dev}")


def _launch(dev, stream, call, *args):
    """``call(*args, stream)`` with device ``dev`` current, on ``stream`` or
    that device's current stream."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(dev, stream, call, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    return call(*args, stream)


def _empty(stream, make=torch.empty):
    """``torch.empty`` (or ``make``) for ``stream``'s use (None: the current
    one's): a block that the current stream has freed may still be in use
    there."""
    if stream is None:
        return make

    def empty(*size, dtype, device):
        on = stream
        if isinstance(stream, int):  # handles 0 and 1 (cudaStreamLegacy): the default stream,
            # of which ExternalStream would make another one
            on = (torch.cuda.default_stream(device) if stream in (0, 1)
                  else torch.cuda.ExternalStream(stream, device))
        with torch.cuda.stream(on):
            return make(*size, dtype=dtype, device=device)
    return empty


def _attention_options(problem, dev, k_pool, k_scales, v_scales, scale_block, logit_cap,
                       alibi_slopes):
    """The run's ``pa_attention_options``, or None if nothing is asked for."""
    if k_scales is None and v_scales is None and scale_block is None:
        if alibi_slopes is None and not logit_cap:
            return None
        scale_block = 0
    else:
        _require(k_scales is not None and v_scales is not None, "k_scales and v_scales together")
        if scale_block is None:
            scale_block = problem.page_size
        _require(scale_block > 0 and problem.page_size % scale_block == 0,
                 "scale_block divides the page")
        heads = problem.num_kv_heads
        _check_scales(k_scales, v_scales,
                      k_pool.numel() // (heads * problem.head_dim) // scale_block, heads, dev)
    if alibi_slopes is not None:
        if not (alibi_slopes.dtype is torch.float32 and alibi_slopes.get_device() == dev
                and alibi_slopes.numel() == problem.num_qo_heads and alibi_slopes.is_contiguous()):
            raise ValueError(f"alibi_slopes: contiguous float32 on cuda:{dev}, one per query head")
    return C.make_options(k_scales=k_scales, v_scales=v_scales, scale_block=scale_block,
                          logit_cap=logit_cap, alibi_slopes=alibi_slopes)


class PagedDecode:
    """Plan once per decode step (host), run once per layer (device).

    ``prefix_len`` > 0 makes a cascade plan: every request first attends to a
    shared prefix of that many tokens (``prefix_indices`` at run time), then
    to its own pages.
    """

    def __init__(self, kv_indptr, last_page_len, *, num_qo_heads, num_kv_heads, page_size,
                 dtype, sm_scale, num_pages, head_dim=128, device=None, num_sms=None,
                 ctas_per_sm=None, min_chunk_tokens=0, prefix_len=0, flags=0,
                 piece_cost_tokens=0, kv_dtype=None, k_scale=1.0, v_scale=1.0,
                 rope_theta=0.0, stream=None):
        self.device = _device(device)
        self._dev = dev_index = self.device.index
        self.dtype = dtype
        self.batch = len(last_page_len)
        self.num_qo_heads, self.head_dim = num_qo_heads, head_dim
        self.prefix_len = prefix_len
        extra = dict(kv_dtype=kv_dtype, k_scale=k_scale, v_scale=v_scale, rope_theta=rope_theta)
        if num_sms is None or ctas_per_sm is None:
            shape = C.make_problem(batch=self.batch, num_qo_heads=num_qo_heads,
                                   num_kv_heads=num_kv_heads, head_dim=head_dim,
                                   page_size=page_size, dtype=dtype, sm_scale=sm_scale,
                                   num_sms=1, ctas_per_sm=1, flags=flags, **extra)
            sms, k = C.pa_problem_schedule(shape, dev_index)
            num_sms = sms if num_sms is None else num_sms
            ctas_per_sm = k if ctas_per_sm is None else ctas_per_sm
        self.problem = C.make_problem(batch=self.batch, num_qo_heads=num_qo_heads,
                                      num_kv_heads=num_kv_heads, head_dim=head_dim,
                                      page_size=page_size, dtype=dtype, sm_scale=sm_scale,
                                      num_sms=num_sms, ctas_per_sm=ctas_per_sm,
                                      min_chunk_tokens=min_chunk_tokens, num_pages=num_pages,
                                      flags=flags, piece_cost_tokens=piece_cost_tokens,
                                      **extra)
        if prefix_len:
            self.plan = C.pa_cascade_plan_create(self.problem, prefix_len, kv_indptr, last_page_len)
        else:
            self.plan = C.pa_plan_create(self.problem, kv_indptr, last_page_len)
        self.workspace_bytes = C.pa_plan_workspace_bytes(self.plan)
        self.workspace = _empty(stream)(max(self.workspace_bytes, 256), dtype=torch.uint8,
                                        device=self.device)
        _launch(self._dev, stream, C.pa_plan_upload, self.plan, self.workspace,
                self.workspace.numel())

    def work_items(self):
        return C.pa_plan_work_items(self.plan)

    def run(self, q, k_pool, v_pool, kv_indices, o=None, lse=None, prefix_indices=None,
            stream=None, *, k_scales=None, v_scales=None, scale_block=None, logit_cap=0.0,
            alibi_slopes=None):
        """``k_scales`` / ``v_scales`` (float32 ``[num_pages * page_size /
        scale_block, num_kv_heads]``, 8-bit pools): a scale for each block of
        ``scale_block`` tokens (default: a page) and kv head, as ``PagedKV``
        writes them.  ``logit_cap``: scores become ``cap * tanh(s / cap)``;
        ``alibi_slopes`` (float32 ``[num_qo_heads]``): scores lose slope *
        distance.  None of them goes with a shared prefix."""
        options = _attention_options(self.problem, self._dev, k_pool, k_scales, v_scales,
                                     scale_block, logit_cap, alibi_slopes)
        _require(options is None or not self.prefix_len, "a cascade run takes no options")
        empty = _empty(stream)
        if o is None:
            o = empty(self.batch, self.num_qo_heads, self.head_dim,
                      dtype=_TORCH_DTYPES[self.dtype], device=self.device)
        if lse is None:
            lse = empty(self.batch, self.num_qo_heads, dtype=torch.float32, device=self.device)
        if self.prefix_len:
            _launch(self._dev, stream, C.pa_cascade_run, self.plan, q, k_pool, v_pool,
                    prefix_indices, kv_indices, o, lse, self.workspace, self.workspace.numel())
        elif options is not None:
            _launch(self._dev, stream, C.pa_run_options, self.plan, options, q, k_pool, v_pool,
                    kv_indices, o, lse, self.workspace, self.workspace.numel())
        else:
            _launch(self._dev, stream, C.pa_run, self.plan, q, k_pool, v_pool, kv_indices, o, lse,
                    self.workspace, self.workspace.numel())
        return o, lse

    def check(self, stream=None) -> int:
        return _launch(self._dev, stream, C.pa_plan_check, self.plan, self.workspace)


class PagedPrefill:
    """Prefill / append attention: plan once per batch of new tokens (host),
    run once per layer (device).  ``qo_indptr`` gives each request's new query
    tokens (rows of q); with ``causal`` they are the last of its keys and
    each sees the keys up to its own position, else every token sees all of
    its request's keys."""

    def __init__(self, qo_indptr, kv_indptr, last_page_len, *, num_qo_heads, num_kv_heads,
                 page_size, dtype, sm_scale, num_pages, causal=True, head_dim=128, device=None,
                 num_sms=None, flags=0, stream=None):
        self.device = _device(device)
        self._dev = self.device.index
        self.dtype = dtype
        self.batch = len(last_page_len)
        self.total_q = int(qo_indptr[-1]) if self.batch else 0
        self.num_qo_heads, self.head_dim = num_qo_heads, head_dim
        # one persistent CTA per SM (ctas_per_sm does not apply to prefill plans)
        if num_sms is None:
            num_sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.problem = C.make_problem(batch=self.batch, num_qo_heads=num_qo_heads,
                                      num_kv_heads=num_kv_heads, head_dim=head_dim,
                                      page_size=page_size, dtype=dtype, sm_scale=sm_scale,
                                      num_sms=num_sms, ctas_per_sm=1, num_pages=num_pages,
                                      flags=flags)
        self.plan = C.pa_prefill_plan_create(self.problem, causal, qo_indptr, kv_indptr,
                                             last_page_len)
        self.workspace_bytes = C.pa_plan_workspace_bytes(self.plan)
        self.workspace = _empty(stream)(max(self.workspace_bytes, 256), dtype=torch.uint8,
                                        device=self.device)
        _launch(self._dev, stream, C.pa_plan_upload, self.plan, self.workspace,
                self.workspace.numel())

    def tiles(self):
        return C.pa_plan_prefill_tiles(self.plan)

    def cta_indptr(self):
        return C.pa_plan_cta_indptr(self.plan)

    def run(self, q, k_pool, v_pool, kv_indices, o=None, lse=None, stream=None, *, logit_cap=0.0,
            alibi_slopes=None):
        """``logit_cap`` and ``alibi_slopes`` as for ``PagedDecode.run``; slopes
        need the causal mask."""
        options = _attention_options(self.problem, self._dev, k_pool, None, None, None,
                                     logit_cap, alibi_slopes)
        empty = _empty(stream)
        if o is None:
            o = empty(self.total_q, self.num_qo_heads, self.head_dim,
                      dtype=_TORCH_DTYPES[self.dtype], device=self.device)
        if lse is None:
            lse = empty(self.total_q, self.num_qo_heads, dtype=torch.float32, device=self.device)
        if options is not None:
            _launch(self._dev, stream, C.pa_prefill_run_options, self.plan, options, q, k_pool,
                    v_pool, kv_indices, o, lse, self.workspace, self.workspace.numel())
        else:
            _launch(self._dev, stream, C.pa_prefill_run, self.plan, q, k_pool, v_pool, kv_indices,
                    o, lse, self.workspace, self.workspace.numel())
        return o, lse

    def check(self, stream=None) -> int:
        return _launch(self._dev, stream, C.pa_plan_check, self.plan, self.workspace)


class PagedKV:
    """Write and read back an 8-bit paged KV cache with one scale for each
    block of ``scale_block`` tokens and kv head: plan once per batch of new
    tokens (host), run once per layer (device).

    The plan covers the last ``qo_indptr[b + 1] - qo_indptr[b]`` tokens of each
    request, whose pages hold them already (lengths after the append).
    ``scale_block`` is a power of two that divides the page (default: a page).
    The pools are ``[num_pages, page_size, num_kv_heads, 128]`` codes
    (``torch.float8_*`` or ``uint8``), the scales float32
    ``[num_pages * page_size / scale_block, num_kv_heads]``; both are read by
    ``PagedDecode.run(..., k_scales=, v_scales=, scale_block=)``.
    """

    def __init__(self, qo_indptr, kv_indptr, last_page_len, *, num_kv_heads, page_size, dtype,
                 kv_dtype, num_pages, scale_block=None, head_dim=128, device=None, flags=0,
                 stream=None):
        self.device = _device(device)
        self._dev = self.device.index
        self.dtype, self.kv_dtype = dtype, kv_dtype
        self.batch = len(last_page_len)
        _require(len(qo_indptr) == self.batch + 1 and len(kv_indptr) == self.batch + 1,
                 "qo_indptr and kv_indptr have batch + 1 entries")
        self.total_q = int(qo_indptr[-1])
        self.total_pages = int(kv_indptr[-1])
        self.num_kv_heads, self.page_size, self.head_dim = num_kv_heads, page_size, head_dim
        self.num_pages = num_pages
        self.scale_block = page_size if scale_block is None else scale_block
        self._row_shape = (self.total_q, num_kv_heads, head_dim)
        self._row_dtype, self._code_dtype = _TORCH_DTYPES[dtype], _KV8_DTYPES[kv_dtype]
        self.problem = C.make_problem(batch=self.batch, num_qo_heads=num_kv_heads,
                                      num_kv_heads=num_kv_heads, head_dim=head_dim,
                                      page_size=page_size, dtype=dtype, sm_scale=1.0, num_sms=1,
                                      ctas_per_sm=1, num_pages=num_pages, flags=flags,
                                      kv_dtype=kv_dtype)
        self.plan = C.pa_kv_plan_create(self.problem, self.scale_block, qo_indptr, kv_indptr,
                                        last_page_len)
        self._pool_elements = num_pages * page_size * num_kv_heads * head_dim
        self._scale_blocks = num_pages * page_size // self.scale_block
        self.workspace_bytes = C.pa_plan_workspace_bytes(self.plan)
        self.workspace = _empty(stream)(max(self.workspace_bytes, 256), dtype=torch.uint8,
                                        device=self.device)
        self.workspace_size = self.workspace.numel()
        _launch(self._dev, stream, C.pa_plan_upload, self.plan, self.workspace,
                self.workspace_size)

    def _check_cache(self, k_pool, v_pool, k_scales, v_scales, kv_indices):
        dev, code, n = self._dev, self._code_dtype, self._pool_elements
        for x in (k_pool, v_pool):
            dtype = x.dtype
            if not ((dtype is code or dtype is torch.uint8) and x.numel() == n
                    and x.get_device() == dev and x.is_contiguous()):
                raise ValueError(f"k_pool and v_pool: contiguous {self.kv_dtype} codes "
                                 f"[{self.num_pages}, {self.page_size}, {self.num_kv_heads}, "
                                 f"{self.head_dim}] on {self.device}")
        _check_scales(k_scales, v_scales, self._scale_blocks, self.num_kv_heads, dev)
        self._check_indices(kv_indices)

    def _check_indices(self, x):
        if not (x.dtype is torch.int32 and x.numel() >= self.total_pages
                and x.get_device() == self._dev and x.is_contiguous()):
            raise ValueError(f"page indices: contiguous int32 on {self.device}, one for each of "
                             f"the plan's {self.total_pages} pages")

    def _row_stride(self, x):
        """Checks 16-bit rows; elements from one to the next."""
        rows, heads, d = self._row_shape
        stride, inner, last = x.stride() if x.dim() == 3 else (0, 0, 0)
        if not (last == 1 and (inner == d or heads == 1) and x.dtype is self._row_dtype
                and x.shape == self._row_shape and x.get_device() == self._dev):
            raise ValueError(f"k and v: {self.dtype} rows {list(self._row_shape)} on "
                             f"{self.device}, the heads of a row packed")
        # a single row has no next one to be apart from
        return stride if rows > 1 else heads * d

    def append(self, k, v, k_pool, v_pool, k_scales, v_scales, kv_indices, stream=None):
        """Quantise the plan's tokens (``k``, ``v``: ``[total_q, num_kv_heads,
        128]``, rows at any stride that is a multiple of 8) into the pools and
        scales, in place.  A block receives tokens through one place of the
        tables only."""
        self._check_cache(k_pool, v_pool, k_scales, v_scales, kv_indices)
        ks, vs = self._row_stride(k), self._row_stride(v)
        _launch(self._dev, stream, C.pa_kv_append, self.plan, k, ks, v, vs, k_pool, v_pool,
                k_scales, v_scales, kv_indices, self.workspace, self.workspace_size)

    def read(self, k_pool, v_pool, k_scales, v_scales, kv_indices, k=None, v=None,
             out_indices=None, stream=None):
        """The plan's tokens in 16 bits: rows ``[total_q, num_kv_heads, 128]``,
        or, with ``out_indices`` (a page of ``k`` / ``v`` for each of the
        plan's pages), pages of the given 16-bit pools ``k`` and ``v``.  A
        token on a bad page (negative, or found out of range by the index
        check) leaves its row of a given ``k`` or ``v`` as it was, and is
        zeros in one that is made here."""
        self._check_cache(k_pool, v_pool, k_scales, v_scales, kv_indices)
        row = self.num_kv_heads * self.head_dim
        out_pages = 0
        if out_indices is not None:
            self._check_indices(out_indices)
            shape = (self.page_size, self.num_kv_heads, self.head_dim)
            for x in (k, v):
                _require(x is not None and x.dtype == _TORCH_DTYPES[self.dtype]
                         and x.device == self.device and x.is_contiguous() and x.dim() == 4
                         and x.shape[1:] == shape,
                         "k and v: contiguous 16-bit pools [pages, page_size, num_kv_heads, 128] "
                         "to unpack into")
            _require(k.shape == v.shape, "k and v pools of the same size")
            ks = vs = row
            out_pages = k.shape[0]
        else:
            ks = vs = row
            # both made here: the kernel writes bad pages' rows, too
            out_pages = C.PA_KV_ZERO_BAD_ROWS if k is None and v is None else 0
            empty = _empty(stream, torch.empty if out_pages else torch.zeros)
            if k is None:
                k = empty(self._row_shape, dtype=self._row_dtype, device=self.device)
            else:
                ks = self._row_stride(k)
            if v is None:
                v = empty(self._row_shape, dtype=self._row_dtype, device=self.device)
            else:
                vs = self._row_stride(v)
        _launch(self._dev, stream, C.pa_kv_read, self.plan, k_pool, v_pool, k_scales, v_scales,
                kv_indices, k, ks, v, vs, out_indices, out_pages, self.workspace,
                self.workspace_size)
        return k, v

    def check(self, stream=None) -> int:
        return _launch(self._dev, stream, C.pa_plan_check, self.plan, self.workspace)
