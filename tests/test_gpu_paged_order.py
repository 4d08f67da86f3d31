"""GPU tests of the order within a stream: the paged calls are set up while the kernel ahead ends, so what
comes before them has to be seen, and what comes behind has to wait, as if every call ended on its own."""
import pytest
import torch

import prefill_only_cascade_gb300 as q

pytestmark = pytest.mark.gpu
DEV, BF, I32 = "cuda", torch.bfloat16, torch.int32


@pytest.fixture(autouse=True)
def no_device_error():
    q.get_device_error()
    yield
    assert q.get_device_error() == q.QUAIL_OK


@pytest.mark.parametrize("lens", [[300, 20], [1 + 41 * i % 250 for i in range(120)], [1500] * 70],
                         ids=["cluster", "pairs", "runs"])
@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
def test_in_order(form, lens):
    B, hkv, hq, d, page, L = len(lens), 8, 32, 64, 16, max(lens)
    width = -(-L // page)
    desc = q.make_paged_desc(B, L, 2 * B * width, page, width, hq, hkv, d, kv_fp8=form == "fp8", kv_fp4=form == "fp4")
    dtype = {"bf16": BF, "fp8": torch.float8_e4m3fn, "fp4": torch.uint8}[form]
    scale = dict(k_scale=None, v_scale=None)
    if form != "bf16":
        scale = {k: torch.full((B, hkv), 4 / (448 if form == "fp8" else 2688), device=DEV) for k in scale}
    T, budget = sum(lens), min(lens) if min(lens) > 8 else 8
    i32 = lambda x: torch.tensor(x, dtype=I32, device=DEV)
    off, zero, n = i32([0, *torch.tensor(lens).cumsum(0).tolist()]), i32([0] * B), i32(lens)
    table = torch.arange(B * width, dtype=I32, device=DEV).view(B, width)
    dst = table[:, :-(-budget // page)].contiguous() + B * width
    base = torch.randn(2, T, hkv, d, generator=torch.Generator().manual_seed(1)).to(DEV)
    q0 = torch.randn(B, hq, d, generator=torch.Generator().manual_seed(2)).to(DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
    ews = torch.empty(q.paged_evict_workspace_size(desc, desc.num_pages), dtype=torch.uint8, device=DEV)

    def run(wait):
        k, v = (torch.zeros(q.paged_pool_shape(desc), dtype=torch.uint8 if form != "bf16" else BF, device=DEV).view(dtype)
                for _ in range(2))
        new = [torch.empty(T, hkv, d, dtype=BF, device=DEV) for _ in range(2)]
        back = [torch.empty(T, hkv, d, dtype=BF, device=DEV) for _ in range(2)]
        qt, out = torch.empty(B, hq, d, dtype=BF, device=DEV), torch.empty(B, hq, d, dtype=BF, device=DEV)
        score = torch.zeros(B, hkv, L, device=DEV)
        kept, fresh = torch.empty(B, hkv, budget, dtype=I32, device=DEV), torch.empty(B, dtype=I32, device=DEV)
        got, step = [], (torch.cuda.synchronize if wait else lambda: None)
        for i in range(6):
            for x, y in zip(new, base):
                x.copy_(y * (0.5 + 0.1 * i))
            qt.copy_(q0 * (1.0 + i))
            step()
            q.paged_kv_append(desc, *new, zero, table, k, v, new_offsets=off, **scale)
            step()
            for x in new:
                x.zero_()                       # behind the append: it has read them
            if form == "fp4" or i % 2 == 0:
                q.paged_kv_read(desc, k, v, zero, table, *back, offsets=off, **scale)
                step()
            q.paged_decode_attn(desc, qt, k, v, table, n, out, ws, score_in=score, score_out=score, **scale)
            step()
            first = out.clone()
            qt.mul_(-1)
            step()
            q.paged_decode_attn(desc, qt, k, v, table, n, out, ws, **scale)
            step()
            q.paged_kv_evict(desc, budget, 2, k, v, table, n, score, dst, k, v, kept, fresh, ews)
            step()
            got += [first, out.clone(), score.clone(), kept.clone(), *(x.clone() for x in back)]
            out.zero_()
            kept.zero_()
        got += [k.view(torch.uint8), v.view(torch.uint8)]
        torch.cuda.synchronize()
        return got

    want = run(True)
    for _ in range(2):
        for i, (a, b) in enumerate(zip(run(False), want)):
            assert torch.equal(a, b), i
