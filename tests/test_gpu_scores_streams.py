"""quail_attn_scores with clusters (few keys, many queries) on several streams at once: the CTAs of
different launches meet on the SMs, each wanting all of an SM's tensor memory."""
import pytest
import torch

import prefill_only_cascade_gb300 as q
from paged_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_clusters_on_streams(d):
    gen = torch.Generator(device=DEV).manual_seed(d)
    hq, hkv, nq, nk = 8, 4, 6000, [300, 90, 256]
    qs = torch.randn(3 * nq, hq, d, generator=gen, device=DEV).bfloat16()
    ks = torch.randn(sum(nk), hkv, d, generator=gen, device=DEV).bfloat16()
    lse = 8 + torch.rand(3 * nq, hq, generator=gen, device=DEV)
    q_off = torch.arange(4, dtype=torch.int32, device=DEV) * nq
    k_off = torch.tensor([0, 300, 390, 646], dtype=torch.int32, device=DEV)

    def call(out, stream=None):
        q.attn_scores(qs, ks, lse, q_off, k_off, out, nq, 300, causal=False, stream=stream)

    want = torch.zeros(3, hkv, 300, device=DEV)
    call(want)
    outs = [torch.zeros_like(want) for _ in range(24)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        call(out, streams[i % 4])
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_OK
    assert float(want.sum()) > 0
    assert all(torch.equal(out, want) for out in outs)
