"""GPU tests of attention over pages of codes whose V scales are near the ends of fp32, by every way of
launching: the quotient of a scale and a sum of weights may be no ordinary number where the output is."""
import numpy as np
import pytest
import torch

import paged_fp4_util
import paged_util
import prefill_only_cascade_gb300 as q

pytestmark = pytest.mark.gpu
WAYS = {   # heads per KV head, KV heads, lengths
    "cluster": (4, 2, [700, 1, 128, 129]),
    "pairs": (4, 7, [1 + 37 * i % 256 for i in range(40)]),
    "pairs of 16": (16, 7, [1 + 37 * i % 256 for i in range(40)]),
    "warps": (16, 7, [1 + 331 * i % 1000 for i in range(100)]),
    "runs": (4, 8, [1025, 4000, 127, 128, 129, 1] * 8),
}


@pytest.mark.parametrize("exponent", [-124, -100, 100])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("form", ["fp8", "fp4"])
def test_v_scales(form, way, exponent):
    group, hkv, lens = WAYS[way]
    d, hq = 128, group * hkv
    util = paged_util if form == "fp8" else paged_fp4_util
    c = paged_util.Cache(lens, hkv, d, 16, True, seed=9) if form == "fp8" else paged_fp4_util.Cache4(lens, hkv, d, 16, seed=9)
    vs = np.ldexp(1 + np.random.default_rng(1).random((len(lens), hkv)), exponent).astype(np.float32)
    c.v_scale = torch.from_numpy(vs).cuda()
    c.vs64 = vs.astype(np.float64)
    c.vs_np = vs
    if form == "fp8" and exponent < 0:
        # values that do not cancel, so that the output is no smaller than they are
        code = c.v.view(torch.uint8)
        code.copy_(torch.where(code == 0x7F, code, code & 0x7E | 0x40))
        c.v64 = c.v.to(torch.float64).cpu().numpy().reshape(c.v64.shape)
    qt = paged_fp4_util.queries(9, len(lens), hq, d)
    q.get_device_error()
    out, lse, _ = util.run_decode(c, qt, hq)
    util.check_decode(c, qt, hq, out, lse, only={0, 1, 3, 28, len(lens) - 1} & set(range(len(lens))))
    assert q.get_device_error() == q.QUAIL_OK


@pytest.mark.parametrize("form", ["fp8", "fp4"])
def test_rows_of_zeros(form):
    """Under the scale that a head of zeros has (1) they come back as zeros, under a scale of 0 as NaN."""
    desc = q.make_paged_desc(1, 20, 2, 16, 2, 2, 2, 64, kv_fp8=form == "fp8", kv_fp4=form == "fp4")
    pools = [torch.full(q.paged_pool_shape(desc), 0x31, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = torch.zeros(20, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = [torch.full_like(rows, 3.0) for _ in range(2)]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    scale = torch.tensor([[1.0, 0.0]], device="cuda")
    kw = dict(k_scale=scale, v_scale=scale)
    q.paged_kv_append(desc, rows, -rows, i32(0), i32(1, 0).view(1, 2), *pools, new_offsets=i32(0, 20), **kw)
    q.paged_kv_read(desc, *pools, i32(0), i32(1, 0).view(1, 2), *out, offsets=i32(0, 20), **kw)
    for x in out:
        assert (x[:, 0] == 0).all() and torch.isnan(x[:, 1].float()).all()
    assert q.get_device_error() == q.QUAIL_OK
