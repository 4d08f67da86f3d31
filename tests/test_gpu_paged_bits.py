"""How many bits the weights of quail_paged_decode_attn keep, and what an infinite V gives."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from paged_util import BF16, DEV, U32

pytestmark = pytest.mark.gpu


def call(qt, k, v, table, lens, scale=0.0, k_scale=None, v_scale=None):
    B, hq, d = qt.shape
    pages, page, hkv, _ = k.shape
    desc = q.make_paged_desc(B, max(lens), pages, page, table.shape[1], hq, hkv, d, scale,
                             k_scale is not None)
    out = torch.empty(B, hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(B, hq, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    q.paged_decode_attn(desc, qt, k, v, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                        out, ws, lse=lse, k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_OK
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,B", [(8, 4), (8, 96)])  # one launch of clusters; runs of warps
def test_weights_keep_their_bits(d, fp8, hkv, B):
    """Three keys a sequence; the first two have the largest score (weight 1 before the division)
    and values that cancel the third's to what 16 bits of them cannot hold. So an error in the
    third's weight shows, which the rounding of the output would hide otherwise.

    The scores are single products: exact but for the scale (2 u), the product (u) and the
    difference (u), so x is off by at most 4 u |x| (|x| <= 4 here), and its weight p by
    ln 2 * 4 u * 4 + 2^-22 (ex2). p itself keeps 24 (bf16 pages) or 22 bits (e4m3: 2 u).
    The sum of the three products, their rescaling and the quotient: 8 u of their magnitudes."""
    gen = torch.Generator().manual_seed(d + B)
    lens, page = [3] * B, 16
    k = torch.zeros(B, page, hkv, d)
    v = torch.zeros(B, page, hkv, d)
    k[:, :2, :, 5] = 2.0
    k[:, 2, :, 5] = 1.0 + torch.randint(0, 8, (B, hkv), generator=gen) / 8
    qt = torch.zeros(B, hkv, d)
    qt[:, :, 5] = (0.25 + torch.rand(B, hkv, generator=gen)).bfloat16().float()
    v[:, 2] = (64 + 150 * torch.rand(B, hkv, d, generator=gen)).mul(
        torch.randint(0, 2, (B, hkv, d), generator=gen) * 2 - 1.0)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    v[:, 2] = v[:, 2].to(dt).float()
    x = (qt[:, :, 5].double() * (k[:, 2, :, 5] - 2.0).double())  # scale 1
    p = torch.exp(x)
    want = p[:, :, None] * v[:, 2].double()
    v[:, 0] = (-want).float().to(dt).float()
    v[:, 1] = (-(want + v[:, 0].double())).float().to(dt).float()
    ones = torch.ones(B, hkv, device=DEV) if fp8 else None
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None]
    got, _ = call(qt.bfloat16().to(DEV), k.to(dt).to(DEV), v.to(dt).to(DEV), table, lens, 1.0, ones, ones)
    total = (2 + p)[:, :, None].numpy()
    ref = (want + v[:, 0].double() + v[:, 1].double()).numpy() / total
    size = (want.abs() + v[:, 0].double().abs() + v[:, 1].double().abs()).numpy() / total
    err = (math.log(2) * 4 * U32 * 4 * math.log2(math.e) + 2.0 ** -22 + 2 * U32) * np.abs(want.numpy()) / total \
        + 8 * U32 * size
    assert (np.abs(got - ref) <= err + BF16 * (np.abs(ref) + err)).all(), \
        np.max(np.abs(got - ref) / (err + BF16 * (np.abs(ref) + err)))

@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [40, 777]), (16, 1, [2, 20000]), (4, 1, [70] * 700)])
def test_infinite_values(hq, hkv, lens):
    """An infinite V that a query sees makes its column infinite (both signs: NaN), as the sum
    of the products does; the other columns are as without it."""
    gen = torch.Generator().manual_seed(3)
    B, d, page = len(lens), 128, 16
    width = -(-max(lens) // page)
    k = torch.randn(B * width, page, hkv, d, generator=gen).bfloat16().to(DEV)
    v = torch.randn(B * width, page, hkv, d, generator=gen).bfloat16().to(DEV)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    qt = (torch.randn(B, hq, d, generator=gen) * 0.3).bfloat16().to(DEV)
    clean, lse0 = call(qt, k, v, table, lens)
    rows = v.view(B, width * page, hkv, d)
    for b, n in enumerate(lens):
        rows[b, n - 1, :, 3] = math.inf
        rows[b, 0, :, 60] = -math.inf
        rows[b, 0, :, 127], rows[b, n - 1, :, 127] = math.inf, -math.inf
        rows[b, n // 2, :, 90] = math.nan
    got, lse = call(qt, k, v, table, lens)
    assert (got[:, :, 3] == math.inf).all() and (got[:, :, 60] == -math.inf).all()
    assert np.isnan(got[:, :, [90, 127]]).all()
    rest = [c for c in range(d) if c not in (3, 60, 90, 127)]
    assert (got[:, :, rest] == clean[:, :, rest]).all() and (lse == lse0).all()


def test_values_without_weight():
    """Keys whose score is -inf have no weight: a finite V of any size adds nothing, also the
    largest."""
    B, d, page, n = 2, 64, 16, 40
    gen = torch.Generator().manual_seed(4)
    k = torch.randn(B * 3, page, 1, d, generator=gen).bfloat16().to(DEV)
    v = torch.randn(B * 3, page, 1, d, generator=gen).bfloat16().to(DEV)
    table = torch.arange(B * 3, dtype=torch.int32, device=DEV).view(B, 3)
    qt = torch.rand(B, 1, d, generator=gen).add(0.1).bfloat16().to(DEV)
    k.view(B, 48, 1, d)[:, 10:n] = -math.inf
    v.view(B, 48, 1, d)[:, 10:n] = 0.0
    want, lse0 = call(qt, k, v, table, [n, n])
    v.view(B, 48, 1, d)[:, 10:n] = torch.finfo(torch.bfloat16).max
    got, lse = call(qt, k, v, table, [n, n])
    assert (got == want).all() and (lse == lse0).all() and np.isfinite(got).all()
