"""quail_attn_scores where a load never arrives (host-side injection: the kernels skip that of a
sequence's first keys): the launch ends by itself with QUAIL_ERR_TIMEOUT, the weights of the keys
concerned stay what they were, the others are right, and the next call is."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged
from paged_util import DEV, f64

pytestmark = pytest.mark.gpu


# queries and keys of two sequences; keys that the CTA without its load was to weigh
@pytest.mark.parametrize("nq,nk,causal,window,lost", [
    ([700, 300], [700, 300], True, 20, 128),      # the window kernel, a CTA per key tile
    ([700, 300], [700, 300], True, 60, 128),      # with two query tiles
    ([700, 300], [700, 300], True, 130, 128),     # with four
    ([600, 400], [600, 400], True, 0, 256),       # the main kernel, a CTA per 256 keys
    ([5000, 4000], [700, 300], False, 0, 256),    # clusters: the last CTA's load is missing
])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_missing_load(nq, nk, causal, window, lost, d, in_place):
    hq, hkv = 4, 2
    gen = torch.Generator().manual_seed(d)
    qs = torch.randn(sum(nq), hq, d, generator=gen).bfloat16()
    ks = torch.randn(sum(nk), hkv, d, generator=gen).bfloat16()
    lse = 7 + torch.rand(sum(nq), hq, generator=gen)
    off = [torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV) for n in (nq, nk)]
    base = torch.rand(2, hkv, 703, generator=gen).to(DEV)
    args = [qs.to(DEV), ks.to(DEV), lse.to(DEV), *off]

    def call():
        out = base.clone() if in_place else torch.full_like(base, -3.0)
        q.attn_scores(*args, out, max(nq), max(nk), causal=causal, window=window,
                      score_in=out if in_place else base)
        return out

    def check(got, first):
        q0 = k0 = 0
        before = f64(base) if in_place else np.full(base.shape, -3.0)
        for s, (a, b) in enumerate(zip(nq, nk)):
            ref = f64(base)[s, :, :b] + paged.scores(
                f64(qs)[q0:q0 + a], f64(ks)[k0:k0 + b], f64(lse)[q0:q0 + a], 1 / math.sqrt(d),
                causal, window)
            assert (got[s, :, :first] == before[s, :, :first]).all()
            assert np.allclose(got[s, :, first:b], ref[:, first:], rtol=1e-4)
            assert (got[s, :, b:] == before[s, :, b:]).all()
            q0, k0 = q0 + a, k0 + b

    q.set_wait_timeout_ns(50_000_000)  # 50 ms
    q.debug_inject(True)
    try:
        out = call()
        assert q.get_device_error() == q.QUAIL_ERR_TIMEOUT
    finally:
        q.debug_inject(False)
        q.set_wait_timeout_ns(0)
    assert q.get_device_error() == q.QUAIL_OK
    check(f64(out), lost)
    out = call()
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_OK
    check(f64(out), 0)
