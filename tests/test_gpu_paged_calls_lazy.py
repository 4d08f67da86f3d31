"""GPU tests of the paged calls on lazy clones: what a call writes is the clone's own, the tensor that it
was cloned from stays as it was, by the native argument checks as by the binding's own."""
import pytest
import torch

import prefill_only_cascade_gb300 as q
from test_gpu_paged_calls import NATIVE, OUTPUTS, U8, arguments

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not hasattr(torch, "_lazy_clone"), reason="no lazy clones")]


def data(t):
    return t.contiguous().view(U8).clone()


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("name", NATIVE)
def test_outputs_that_are_lazy_clones(name, form, native):
    written = OUTPUTS[name] + (("workspace",) if name in ("decode", "evict") else ())
    kw = {} if native else dict(stream=torch.cuda.current_stream())
    filled = arguments(form)
    q.paged_kv_append(**filled["append"])          # pages with rows in them
    pools = [filled["append"][x].clone() for x in ("k_pages", "v_pages")]
    args = arguments(form)[name]
    if name != "append":
        args["k_pages"], args["v_pages"] = pools
    torch.manual_seed(0)
    for x in written:
        args[x].view(U8).copy_(torch.randint(0, 120, args[x].view(U8).shape, dtype=U8, device="cuda"))
    if name == "evict":
        args["score"].copy_(torch.rand(args["score"].shape, device="cuda"))
    first = {x: args[x].clone() for x in written}
    before = {x: data(args[x]) for x in written}
    lazy = {**args, **{x: torch._lazy_clone(args[x]) for x in written}}
    NATIVE[name](**lazy, **kw)
    for x in written:
        assert torch.equal(data(args[x]), before[x]), x
    plain = {**args, **first}
    NATIVE[name](**plain, **kw)
    for x in OUTPUTS[name]:
        assert torch.equal(data(lazy[x]), data(plain[x])), x
        assert not torch.equal(data(lazy[x]), before[x]), x
    assert q.get_device_error() == q.QUAIL_OK


@pytest.mark.skipif(q._calls is None, reason="built without PyTorch's or Python's headers")
@pytest.mark.parametrize("name", NATIVE)
def test_lazy_clones_go_the_native_way(name):
    args = arguments("fp4")[name]
    lazy = {k: torch._lazy_clone(v) if isinstance(v, torch.Tensor) else v for k, v in args.items()}
    assert getattr(q._calls, name)(*lazy.values()) == q.QUAIL_OK
    assert q.get_device_error() == q.QUAIL_OK
