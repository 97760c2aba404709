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
