"""GPU parity of eviction from 4-bit pages, bit for bit: the kept tokens' codes and block scales at
their new places, everything else as it was; and a cut cache attended to."""
import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import fp4, paged
from paged_fp4_util import Cache4, check_decode, queries, run_decode
from paged_util import DEV, block_table

pytestmark = pytest.mark.gpu


def evict(c, score, budget, recent, same=False, table=None, max_len=None):
    """dst: pages of another pool, or fresh ones of the cache's own; all destination bytes are 0x55."""
    B, hkv = len(c.lens), c.hkv
    fresh = [min(n, budget) for n in c.lens]
    t, pages = block_table(fresh, c.page, np.random.default_rng(1), width=-(-budget // c.page))
    head = c.k.shape[2]
    empty = lambda n: torch.full((n, hkv, head), 0x55, dtype=torch.uint8, device=DEV)
    if same:
        t = np.where(t >= 0, t + c.pages, t).astype(np.int32)
        c.k, c.v = (torch.cat([x, empty(pages)]) for x in (c.k, c.v))
        c.pages += pages
        k_dst, v_dst = c.k, c.v
    else:
        k_dst, v_dst = empty(pages), empty(pages)
    t = t if table is None else table(t)
    desc = c.desc(hkv, max_len)
    kept = torch.full((B, hkv, budget), -9, dtype=torch.int32, device=DEV)
    new = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    ws = torch.full((q.paged_evict_workspace_size(desc, k_dst.shape[0]),), 0xA5, dtype=torch.uint8, device=DEV)
    q.paged_kv_evict(desc, budget, recent, c.k, c.v, c.table, c.seq_lens, score.to(DEV),
                     torch.from_numpy(t).to(DEV), k_dst, v_dst, kept, new, ws)
    return kept.cpu().numpy(), new.cpu().numpy(), k_dst, v_dst, t


def check(c, score, budget, recent, got, same=False):
    kept, new, k_dst, v_dst, table = got
    s = score.numpy()
    for src, dst in ((c.k_np, k_dst), (c.v_np, v_dst)):
        codes, blocks = fp4.parts(src, c.page, c.d)
        n_dst = dst.shape[0]
        base = np.full((n_dst, c.hkv, c.k_np.shape[2]), 0x55, np.uint8)
        if same:
            base[:len(src)] = src
        to_codes, to_blocks = (x.copy() for x in fp4.parts(base, c.page, c.d))
        for b, n in enumerate(c.lens):
            m = min(n, budget)
            assert new[b] == m
            for g in range(c.hkv):
                want = paged.evict(s[b, g], n, budget, recent)
                np.testing.assert_array_equal(kept[b, g, :m], want)
                i = np.arange(m)
                a, z = c.table_np[b, want // c.page], table[b, i // c.page]
                to_codes[z, g, i % c.page] = codes[a, g, want % c.page]
                to_blocks[z, g, i % c.page] = blocks[a, g, want % c.page]
        np.testing.assert_array_equal(dst.cpu().numpy(), fp4.join(to_codes, to_blocks))


@pytest.mark.parametrize("lens,budget,recent,hkv,d,page", [
    ([0, 1, 5, 40, 41, 100, 333, 1000, 2049], 40, 8, 2, 128, 16),      # one launch
    ([10, 90, 300], 50, 50, 3, 64, 32), ([1, 2, 700], 1, 0, 2, 64, 16),
    ([5, 60, 64], 64, 3, 8, 128, 64), ([16000, 900, 1024], 1000, 990, 1, 64, 256),
    ([600, 2048], 513, 100, 2, 128, 16),                               # two launches
    ([5000] * 12, 1000, 16, 4, 128, 128), ([70000], 3000, 64, 1, 64, 64), ([0, 0], 16, 4, 2, 128, 16),
])
@pytest.mark.parametrize("same", [False, True])
def test_eviction(lens, budget, recent, hkv, d, page, same):
    c = Cache4(lens, hkv, d, page, seed=3, width=max(1, -(-max(max(lens), 1) // page)))
    score = torch.randn(len(lens), hkv, max(max(lens), 1), generator=torch.Generator().manual_seed(2))
    got = evict(c, score, budget, recent, same)
    assert q.get_device_error() == q.QUAIL_OK
    check(c, score, budget, recent, got, same)


def test_bad_destinations_are_not_written():
    """A destination page that two sequences name is written by neither; the third's are whole."""
    c = Cache4([200, 200, 200], 2, 128, 16, seed=5)
    score = torch.randn(3, 2, 200, generator=torch.Generator().manual_seed(5))

    def twice(t):
        t[1, 1] = t[0, 2]
        return t
    kept, new, k_dst, v_dst, table = evict(c, score, 64, 8, table=twice)
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    assert list(new) == [-1, -1, 64]
    for dst in (k_dst, v_dst):
        assert (dst[int(table[0, 2])].cpu().numpy() == 0x55).all()
    c.lens = [0, 0, 200]
    codes, blocks = fp4.parts(c.k_np, 16, 128)
    to_codes, to_blocks = fp4.parts(k_dst.cpu().numpy(), 16, 128)
    for g in range(2):
        want = paged.evict(score[2, g].numpy(), 200, 64, 8)
        i = np.arange(64)
        np.testing.assert_array_equal(to_codes[table[2, i // 16], g, i % 16],
                                      codes[c.table_np[2, want // 16], g, want % 16])
        np.testing.assert_array_equal(to_blocks[table[2, i // 16], g, i % 16],
                                      blocks[c.table_np[2, want // 16], g, want % 16])


@pytest.mark.parametrize("lens", [[900, 300], [6000, 2500, 100]])
def test_scored_cut_and_attended_to(lens):
    """The weights of an attention step decide what stays; the cut cache is attended to."""
    hq, hkv, d, page, budget = 8, 2, 128, 16, 256
    c = Cache4(lens, hkv, d, page, seed=6)
    B = len(lens)
    _, _, score = run_decode(c, queries(6, B, hq, d), hq, True)
    score = score[:, :, :max(lens)].contiguous()
    host = score.cpu()
    kept, new, k_dst, v_dst, table = evict(c, host, budget, 32)
    check(c, host, budget, 32, (kept, new, k_dst, v_dst, table))
    cut = Cache4.__new__(Cache4)
    cut.__dict__.update(c.__dict__)
    cut.lens, cut.pages, cut.table_np = [min(n, budget) for n in lens], k_dst.shape[0], table
    cut.k, cut.v, cut.table = k_dst, v_dst, torch.from_numpy(table).to(DEV)
    cut.k_np, cut.v_np = k_dst.cpu().numpy(), v_dst.cpu().numpy()
    cut.seq_lens = torch.from_numpy(new).to(DEV)
    qt = queries(7, B, hq, d)
    check_decode(cut, qt, hq, *run_decode(cut, qt, hq)[:2])
    assert q.get_device_error() == q.QUAIL_OK
