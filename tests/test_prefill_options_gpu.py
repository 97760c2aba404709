"""Prefill with options where its arithmetic is at its limits."""
import pytest
import torch

from parity import to_np
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
