"""GPU test of eviction by the native argument checks and by the binding's own: the same call, whatever its
widths, budgets and outputs."""
import pytest
import torch

import prefill_only_cascade_gb300 as q
from test_gpu_paged_calls import OUTPUTS, U8, arguments

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(q._calls is None, reason="built without PyTorch's or Python's headers")]


@pytest.mark.parametrize("budget,recent", [(20, 4), (7, 0), (16, 16), (30, 1), (1, 1)])
@pytest.mark.parametrize("width", [40, 57])
@pytest.mark.parametrize("scored", [True, False])
@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
def test_both_ways_evict_the_same(form, scored, width, budget, recent):
    calls = arguments(form)
    q.paged_kv_append(**calls["append"])
    args = calls["evict"]
    args["k_pages"], args["v_pages"] = calls["append"]["k_pages"], calls["append"]["v_pages"]
    gen = torch.Generator().manual_seed(budget)
    args["score"] = torch.rand(2, 2, width, generator=gen).cuda()
    args["budget"], args["recent"] = budget, recent
    args["kept"] = torch.zeros(2, 2, budget, dtype=torch.int32, device="cuda")
    args["score_out"] = torch.zeros(2, 2, budget + 3, device="cuda") if scored else None
    got = []
    for native in (True, False):
        these = dict(args)
        for x in OUTPUTS["evict"] + ("workspace",):
            if args[x] is not None:
                these[x] = torch.full_like(args[x].view(U8), 0x5A).view(args[x].dtype)
        if native:
            assert q._calls.evict(*these.values()) == q.QUAIL_OK
        else:
            q.paged_kv_evict(**these, stream=torch.cuda.current_stream())
        got.append({x: these[x].view(U8) for x in OUTPUTS["evict"] if args[x] is not None})
        # every value of these is written
        fresh = these["new_lens"].tolist()
        assert fresh == [min(n, budget) for n in (40, 20)]
        assert these["kept"][0, 0].tolist() == sorted(set(these["kept"][0, 0].tolist()))
    assert got[0].keys() == got[1].keys()
    for x in got[0]:
        assert torch.equal(got[0][x], got[1][x]), x
    assert q.get_device_error() == q.QUAIL_OK
