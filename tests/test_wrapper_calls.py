"""How the wrapper's calls reach the library: device and stream of every run,
checked on the CPU with the C call replaced."""
import contextlib
import types

import pytest
import torch

CALLS = [("pa_run", dict()), ("pa_run_options", dict(logit_cap=30.0)),
         ("pa_cascade_run", dict(prefix_indices=5)),
         ("pa_prefill_run", dict()), ("pa_prefill_run_options", dict(logit_cap=30.0))]


@pytest.fixture
def device(monkeypatch):
    """Two devices, 0 current; a device's current stream is 100 + its index."""
    state = types.SimpleNamespace(current=0)

    @contextlib.contextmanager
    def use(index):
        before, state.current = state.current, index
        yield
        state.current = before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index,
                        raising=False)
    return state


@pytest.mark.parametrize("stream", [None, 77])
@pytest.mark.parametrize("dev", [0, 1])
@pytest.mark.parametrize("name,kw", CALLS)
def test_runs_go_to_the_plans_device(name, kw, dev, stream, device, monkeypatch):
    from serving_attention_paged_b200 import pagedattn as C
    from serving_attention_paged_b200 import wrapper
    seen = []
    monkeypatch.setattr(C, name, lambda *a: seen.append((device.current, C._stream(a[-1]))))
    kind = wrapper.PagedPrefill if "prefill" in name else wrapper.PagedDecode
    plan = object.__new__(kind)
    plan._dev, plan.device, plan.plan = dev, torch.device("cuda", dev), None
    plan.problem = types.SimpleNamespace(page_size=16)
    plan.prefix_len = 16 if "cascade" in name else 0
    plan.workspace = torch.empty(256, dtype=torch.uint8)
    plan.run(1, 2, 3, 4, o=6, lse=7, stream=stream, **kw)
    assert seen == [(dev, 100 + dev if stream is None else stream)]
    assert device.current == 0


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [0, 1, "default", "side"])
def test_outputs_come_from_the_given_handles_pool(handle):
    """A raw handle, the legacy default stream's (0, or cudaStreamLegacy = 1)
    included: outputs are blocks of that stream's memory, not of some other
    stream's, on which earlier work may still use them."""
    from serving_attention_paged_b200 import workloads as W
    from serving_attention_paged_b200.wrapper import PagedDecode
    w = W.make_workload("handles", [40, 17], num_qo_heads=8, num_kv_heads=2, page_size=16,
                        dtype="f16", seed=3)
    t = {k: v.cuda() for k, v in w.materialize().items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle = {"default": torch.cuda.default_stream().cuda_stream,
              "side": side.cuda_stream}.get(handle, handle)
    pd = PagedDecode(w.kv_indptr, w.last_page_len, num_qo_heads=8, num_kv_heads=2, page_size=16,
                     dtype="f16", sm_scale=w.sm_scale, num_pages=w.num_pages, stream=handle)
    outputs = pd.run(t["q"], t["k_pool"], t["v_pool"], t["kv_indices"], stream=handle)
    torch.cuda.synchronize()
    assert pd.check(stream=handle) == -1
    want = side.cuda_stream if handle == side.cuda_stream else 0
    for x in (*outputs, pd.workspace):
        owner = [s["stream"] for s in torch.cuda.memory_snapshot()
                 if s["address"] <= x.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [want]
