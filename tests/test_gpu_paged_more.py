"""Paths of the paged calls that the sizes of the other tests do not reach."""
import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged
from paged_util import DEV, Cache, check_decode, run_decode
from test_gpu_paged import ok, queries
from test_gpu_paged_evict import raw, run, scores_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,B", [(8, 8, 256), (16, 2, 1024), (4, 1, 2048)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_in_several_chunks(hq, hkv, B, fp8, in_place):
    """2,048 (sequence, head)s with max_seq_len past 4,096: a block forms the weights of several
    runs of 1,024 keys, one after the other."""
    rng = np.random.default_rng(hq)
    lens = rng.integers(0, 40, B).tolist()
    some = {0: 1, 1: 1024, 2: 1025, 3: 0, B // 2: 4097, B // 2 + 1: 2049, B - 2: 5999, B - 1: 6000}
    for b, n in some.items():
        lens[b] = n
    cache = Cache(lens, hkv, 64, 64, fp8, seed=B)
    qt = queries(B, hq, 64, seed=hq)
    base = torch.rand(B, hkv, 6005, device=DEV)
    for b, n in enumerate(lens):
        base[b, :, n:] = -3.0
    score = base.clone() if in_place else torch.full_like(base, -3.0)
    out, lse, _ = run_decode(cache, qt, hq, True, score if in_place else base, max_len=6000,
                             score_out=score)
    ok()
    check_decode(cache, qt, hq, out, lse, score, base, only=set(some) | {4, B - 3})
    for b, n in enumerate(lens):
        assert (score[b, :, n:] == -3.0).all()


@pytest.mark.parametrize("most", [200, 3000, 20000])  # one launch; of clusters; select and copy
@pytest.mark.parametrize("where", ["twice", "itself", "held", "outside"])
@pytest.mark.parametrize("fp8", [False, True])
def test_contested_destination_pages_stay_as_they_were(where, most, fp8):
    """Two claims of a page (by two sequences or by one), or a page that a sequence holds: K and V
    of it are untouched. The other pages of such a sequence may be written."""
    cache = Cache([200, 150, 90], 2, 128, 16, fp8, width=-(-most // 16))
    score = scores_for(cache.lens, 2, most, "normal")
    pages = cache.pages
    kept = (cache.k.clone(), cache.v.clone())
    contested = []

    def spoil(table):
        table = table.copy()
        if where == "twice":
            table[0, 2] = table[1, 3]
            contested.append(int(table[1, 3]))
        elif where == "itself":
            table[1, 0] = table[1, 2]
            contested.append(int(table[1, 2]))
        elif where == "held":
            table[1, 3] = cache.table_np[2, 1]
        else:
            table[1, 0] = cache.pages
        return table

    got = run(cache, score, 64, 8, dst="same", dst_table=spoil, max_len=most)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    table, hit = got[5], ({0, 1} if where == "twice" else {1})
    for now, before in zip((cache.k, cache.v), kept):
        assert torch.equal(now[:pages].view(torch.uint8), before.view(torch.uint8))
        for p in contested:
            assert (now[p].view(torch.uint8) == 0).all()
    # the other sequences' rows, in K and V
    for b in set(range(3)) - hit:
        assert int(got[1][b]) == min(cache.lens[b], 64)
        for g in range(2):
            want = paged.evict(score[b, g].numpy(), cache.lens[b], 64, 8)
            src = paged.slots(cache.table_np[b], want, 16)
            dst = paged.slots(table[b], np.arange(len(want)), 16)
            for now, before in zip((cache.k, cache.v), kept):
                np.testing.assert_array_equal(raw(now)[dst, g], raw(before)[src, g])
