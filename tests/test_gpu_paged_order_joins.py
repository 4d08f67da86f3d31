"""GPU tests of the paged calls behind work of other streams and behind copies, which have no kernel ahead to
be set up beside: called, and captured into a graph with several branches."""
import pytest
import torch

import prefill_only_cascade_gb300 as q

pytestmark = pytest.mark.gpu
DEV, BF, I32 = "cuda", torch.bfloat16, torch.int32


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("lens", [[300, 20], [1 + 41 * i % 250 for i in range(120)], [1500] * 70],
                         ids=["cluster", "pairs", "runs"])
@pytest.mark.parametrize("form", ["bf16", "fp8", "fp4"])
def test_behind_other_streams(form, lens, captured):
    B, hkv, hq, d, page, L = len(lens), 8, 32, 64, 16, max(lens)
    width = -(-L // page)
    desc = q.make_paged_desc(B, L, B * width, page, width, hq, hkv, d, kv_fp8=form == "fp8", kv_fp4=form == "fp4")
    dtype = {"bf16": BF, "fp8": torch.float8_e4m3fn, "fp4": torch.uint8}[form]
    scale = dict(k_scale=None, v_scale=None)
    if form != "bf16":
        scale = {k: torch.full((B, hkv), 4 / (448 if form == "fp8" else 2688), device=DEV) for k in scale}
    T, budget = sum(lens), 16
    i32 = lambda x: torch.tensor(x, dtype=I32, device=DEV)
    off, zero, n = i32([0, *torch.tensor(lens).cumsum(0).tolist()]), i32([0] * B), i32(lens)
    table = torch.arange(B * width, dtype=I32, device=DEV).view(B, width)
    ktab = torch.zeros_like(table)
    gen = torch.Generator().manual_seed(3)
    src = [torch.randn(T, hkv, d, generator=gen).to(BF).to(DEV) for _ in range(2)]
    q0 = torch.randn(B, hq, d, generator=gen).to(BF).to(DEV)
    new, back = ([torch.zeros_like(x) for x in src] for _ in range(2))
    qt, out, other = torch.zeros_like(q0), torch.zeros_like(q0), torch.zeros_like(q0)
    k, v = (torch.zeros(q.paged_pool_shape(desc), dtype=dtype if form != "fp8" else torch.uint8, device=DEV).view(dtype)
            for _ in range(2))
    dk, dv = (torch.zeros_like(k.view(torch.uint8)).view(dtype) for _ in range(2))
    score = torch.zeros(B, hkv, L, device=DEV)
    kept, fresh = torch.zeros(B, hkv, budget, dtype=I32, device=DEV), torch.zeros(B, dtype=I32, device=DEV)
    dst = torch.arange(B, dtype=I32, device=DEV).view(B, 1)
    ws, ws2 = (torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV) for _ in range(2))
    ews = torch.empty(q.paged_evict_workspace_size(desc, desc.num_pages), dtype=torch.uint8, device=DEV)
    sides = [torch.cuda.Stream() for _ in range(2)]

    def step(wait):
        """Each call waits for a copy, a fill or a kernel of another stream as well as for its own."""
        main = torch.cuda.current_stream()
        for s in sides:
            s.wait_stream(main)
        with torch.cuda.stream(sides[0]):
            for x, y in zip(new, src):
                x.copy_(y)                       # a copy
            ktab.copy_(table)
        with torch.cuda.stream(sides[1]):
            torch.add(q0, 0, out=qt)             # a kernel
        main.wait_stream(sides[0])
        wait()
        q.paged_kv_append(desc, *new, zero, ktab, k, v, new_offsets=off, **scale)
        wait()
        main.wait_stream(sides[1])
        q.paged_decode_attn(desc, qt, k, v, ktab, n, out, ws, score_out=score, **scale)
        wait()
        sides[0].wait_stream(main)
        with torch.cuda.stream(sides[0]):        # beside the next calls
            q.paged_decode_attn(desc, qt, k, v, ktab, n, other, ws2, **scale)
        q.paged_kv_read(desc, k, v, zero, ktab, *back, offsets=off, **scale)
        wait()
        q.paged_kv_evict(desc, budget, 2, k, v, ktab, n, score, dst, dk, dv, kept, fresh, ews)
        wait()
        main.wait_stream(sides[0])
        wait()
        for x in new:
            x.zero_()
        qt.zero_()
        ktab.zero_()

    outputs = (out, other, score, kept, fresh, *back, k.view(torch.uint8), v.view(torch.uint8), dk.view(torch.uint8),
               dv.view(torch.uint8))

    def clear():
        for x in outputs:
            x.zero_()
        torch.cuda.synchronize()

    q.get_device_error()
    clear()
    step(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [x.clone() for x in outputs]
    assert torch.equal(out, other) and out.abs().sum() > 0
    run = lambda: step(lambda: None)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        run = graph.replay
    for _ in range(5):
        clear()
        run()
        torch.cuda.synchronize()
        assert q.get_device_error() == q.QUAIL_OK
        for i, (a, b) in enumerate(zip(outputs, want)):
            assert torch.equal(a, b), i
