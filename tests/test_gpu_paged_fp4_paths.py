"""GPU tests of the ways in which attention over 4-bit pages is launched (a cluster, a warp or a run of
tiles for the sequences' heads), against the oracle: every group of heads, pages smaller and larger than
a tile, what is bad in the middle, loads that never arrive; pools past 2^31 bytes; two calls at once."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import fp4, paged
from paged_fp4_util import Cache4, check_decode, queries, run_decode
from paged_util import BF16, DEV, f64

pytestmark = pytest.mark.gpu
DEVICE_BOUNDS = q.QUAIL_ERR_DEVICE_BOUNDS


@pytest.fixture(autouse=True)
def no_device_error():
    q.get_device_error()
    yield
    assert q.get_device_error() == q.QUAIL_OK


# lengths for each way (d = 128; half the steps at d = 64): one launch of clusters, a warp per
# (sequence, head) (few enough for two with 16 heads, and more), runs of warps, runs of CTAs
WAYS = {
    "cluster": [700, 1, 128, 0, 129],
    "pairs": [1 + 37 * i % 256 for i in range(99)] + [0, 256, 32, 33, 31],
    "many pairs": [1 + 5 * i % 64 for i in range(290)] + [0, 64],
    "warps": [1 + 331 * i % 1000 for i in range(100)] + [0, 1024, 257],
    "runs": [1025, 0, 4000, 127, 128, 129, 1, 2047, 2048, 3333] * 8,
}


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("group,d", [(1, 128), (2, 64), (4, 128), (4, 64), (8, 128), (8, 64), (16, 128), (16, 64)])
@pytest.mark.parametrize("way", WAYS)
def test_ways(way, group, d, page):
    hkv = 2 if way == "cluster" else 7
    lens = WAYS[way]
    c = Cache4(lens, hkv, d, page, seed=group + page)
    hq = group * hkv
    qt = queries(group, len(lens), hq, d, scale=1.5)
    score_in = torch.rand(len(lens), hkv, max(lens) + 5, device=DEV)
    plain = run_decode(c, qt, hq)
    scored = run_decode(c, qt, hq, True, score_in)
    some = {0, 1, 2, 3, 4, len(lens) - 4, len(lens) - 2, len(lens) - 1} | set(range(0, len(lens), 23))
    check_decode(c, qt, hq, *plain[:2], only=some)
    check_decode(c, qt, hq, *scored, score_in, only=some)
    assert torch.equal(plain[0], scored[0])
    again = run_decode(c, qt, hq, True, score_in)
    assert all(torch.equal(a, b) for a, b in zip(scored, again))


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("way", WAYS)
def test_bad_pages_and_lengths_in_the_middle(way, page):
    """NaN and a report for what is bad, everything else as it would be."""
    lens = list(WAYS[way])
    hkv, hq, d = (2, 8, 128) if way == "cluster" else (7, 28, 128)
    c = Cache4(lens, hkv, d, page, seed=3)
    qt = queries(3, len(lens), hq, d)
    table, seq_lens = c.table.clone(), c.seq_lens.clone()
    deep = int(np.argmax(lens))
    table[deep, (lens[deep] - 1) // page // 2] = -7
    table[0, 0] = c.pages
    seq_lens[1] = max(lens) + 1
    seq_lens[4] = -1
    bad = {deep, 0, 1, 4}
    desc = c.desc(hq)
    out = torch.full((len(lens), hq, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(lens), hq), 3.0, device=DEV)
    score = torch.full((len(lens), hkv, max(lens)), -3.0, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    for scored in (False, True):
        q.paged_decode_attn(desc, qt, c.k, c.v, table, seq_lens, out, ws, lse=lse,
                            score_out=score if scored else None, **kw)
        assert q.get_device_error() == DEVICE_BOUNDS
        o, l_ = f64(out), f64(lse)
        for b in bad:
            assert np.isnan(o[b]).all() and np.isnan(l_[b]).all(), b
        good = set(range(len(lens))) - bad
        assert np.isfinite(o[sorted(good)]).all()
        check_decode(c, qt, hq, out, lse, only={b for b in good if b < 12})
    s = f64(score)
    assert (s[1] == -3).all() and (s[4] == -3).all()      # no keys of theirs
    for b in (0, deep):
        assert (s[b, :, lens[b]:] == -3).all()


@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("way", WAYS)
def test_loads_that_never_arrive(way, group):
    """The wait runs out, the call ends, its results are NaN, and the next call is right."""
    lens = WAYS[way]
    hkv = 2 if way == "cluster" else 7
    c = Cache4(lens, hkv, 128, 64, seed=5)
    hq = group * hkv
    qt = queries(5, len(lens), hq, 128)
    q.set_wait_timeout_ns(5_000_000)  # 5 ms
    q.debug_inject(True)
    try:
        out, lse, _ = run_decode(c, qt, hq)
        assert q.get_device_error() == q.QUAIL_ERR_TIMEOUT
    finally:
        q.debug_inject(False)
        q.set_wait_timeout_ns(0)
    some = np.array(lens) > 0
    assert np.isnan(f64(out)[some]).all() and np.isnan(f64(lse)[some]).all()
    assert (f64(out)[~some] == 0).all()
    out, lse, _ = run_decode(c, qt, hq)
    check_decode(c, qt, hq, out, lse, only={0, 1, 2, 3})


def test_pools_past_32_bits():
    """Rows, attention and eviction in the last pages of pools of 2.4 GB."""
    hkv, hq, d, page, pages, lens = 8, 32, 128, 256, 16400, [700, 300]
    desc = q.make_paged_desc(2, 1024, pages, page, 4, hq, hkv, d, kv_fp4=True)
    pools = [torch.empty(q.paged_pool_shape(desc), dtype=torch.uint8, device=DEV) for _ in range(2)]
    assert pools[0].numel() > 2 ** 31
    table = torch.full((2, 4), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([pages - 1, 3, pages - 2])
    table[1, :2] = torch.tensor([pages - 5, pages - 4])
    table = table.to(DEV)
    new = [queries(i, sum(lens), hkv, d) for i in range(2)]
    scale = [torch.full((2, hkv), float(x.abs().max()) / 2688, device=DEV) for x in new]
    kw = dict(k_scale=scale[0], v_scale=scale[1])
    off = torch.tensor([0, 700, 1000], dtype=torch.int32, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    q.paged_kv_append(desc, *new, zero, table, *pools, new_offsets=off, **kw)
    back = [torch.empty_like(x) for x in new]
    q.paged_kv_read(desc, *pools, zero, table, *back, offsets=off, **kw)
    rows = []
    for x, got, s in zip(new, back, scale):
        codes, blocks = fp4.quantise(x.float().cpu().numpy(), f64(s)[0])
        rows.append(fp4.values(codes, blocks, f64(s)[0]))
        ref = torch.from_numpy(rows[-1].astype(np.float32)).bfloat16()
        np.testing.assert_array_equal(f64(got), f64(ref))
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qt = queries(9, 2, hq, d)
    out, lse = torch.empty(2, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(2, hq, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    q.paged_decode_attn(desc, qt, *pools, table, seq_lens, out, ws, lse=lse, **kw)
    for b, at in enumerate((slice(0, 700), slice(700, 1000))):
        ref, ref_lse, _ = paged.decode(f64(qt)[b], rows[0][at], rows[1][at], 1 / math.sqrt(d))
        np.testing.assert_allclose(f64(out)[b], ref, atol=1e-5, rtol=2 * BF16)
        np.testing.assert_allclose(f64(lse)[b], ref_lse, atol=2e-5)
    # the first 100 of sequence 0 and all that stay of sequence 1 to other late pages of the pool
    score = torch.zeros(2, hkv, 1024, device=DEV)
    score[:, :, :100] = 1.0
    dst = torch.tensor([[pages - 7], [pages - 9]], dtype=torch.int32, device=DEV)
    kept = torch.empty(2, hkv, 100, dtype=torch.int32, device=DEV)
    n = torch.empty(2, dtype=torch.int32, device=DEV)
    ews = torch.empty(q.paged_evict_workspace_size(desc, pages), dtype=torch.uint8, device=DEV)
    q.paged_kv_evict(desc, 100, 0, *pools, table, seq_lens, score, dst, *pools, kept, n, ews)
    assert n.tolist() == [100, 100]
    short = [torch.empty(200, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ddesc = q.make_paged_desc(2, 100, pages, page, 1, hq, hkv, d, kv_fp4=True)
    q.paged_kv_read(ddesc, *pools, zero, dst, *short, offsets=torch.tensor([0, 100, 200], dtype=torch.int32,
                                                                          device=DEV), **kw)
    for got, all_ in zip(short, back):
        assert torch.equal(got[:100], all_[:100]) and torch.equal(got[100:], all_[700:800])


@pytest.mark.parametrize("way", WAYS)
def test_two_calls_at_once(way):
    lens = WAYS[way]
    hkv = 2 if way == "cluster" else 7
    c = Cache4(lens, hkv, 128, 32, seed=6)
    hq = 4 * hkv
    desc = c.desc(hq)
    qs = [queries(6 + i, len(lens), hq, 128) for i in range(2)]
    want = [run_decode(c, x, hq)[0] for x in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    spaces = [torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for s, x, out, ws in zip(streams, qs, outs, spaces):
            q.paged_decode_attn(desc, x, c.k, c.v, c.table, c.seq_lens, out[i], ws, k_scale=c.k_scale,
                                v_scale=c.v_scale, stream=s)
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in out)


@pytest.mark.parametrize("kind", ["any", "powers of two", "near powers of two", "few bits", "eighths"])
@pytest.mark.parametrize("d", [64, 128])
def test_append_next_to_the_borders(kind, d):
    """Quotients that fall next to a border between codes, or between block scales, for scales whose
    products with a block scale are short, long and in between: bit for bit."""
    rng = np.random.default_rng(len(kind) + d)
    B, hkv, page, n = 32, 4, 32, 32
    S = (10.0 ** rng.uniform(-6, 3, (B, hkv))).astype(np.float32)
    if kind == "powers of two":
        S = (2.0 ** rng.integers(-20, 10, (B, hkv))).astype(np.float32)
    elif kind == "near powers of two":
        S = (2.0 ** rng.integers(-20, 10, (B, hkv)) * (1 + rng.integers(-40, 41, (B, hkv)) * 2.0 ** -23)).astype(np.float32)
    elif kind == "few bits":
        S = ((S.view(np.uint32) & 0xFFFF0000) + rng.integers(-20, 21, S.shape).astype(np.uint32)).view(np.float32)
    each = np.repeat(S, n, 0)[..., None].astype(np.float64)
    x = rng.normal(size=(B * n, hkv, d)) * 10.0 ** rng.uniform(-1, 4, (B * n, hkv, 1))
    if kind == "eighths":
        x = np.round(rng.uniform(-56, 56, (B * n, hkv, d))) / 8 * 2.0 ** rng.integers(-8, 9, (B * n, hkv, d // 16)).repeat(16, -1)
    new = torch.from_numpy((x * each).astype(np.float32)).bfloat16()
    desc = q.make_paged_desc(B, page, B, page, 1, hkv, hkv, d, kv_fp4=True)
    pools = [torch.zeros(q.paged_pool_shape(desc), dtype=torch.uint8, device=DEV) for _ in range(2)]
    table = torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1)
    off = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    s = torch.from_numpy(S).to(DEV)
    q.paged_kv_append(desc, new.to(DEV), (-new).to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV), table,
                      *pools, new_offsets=off, k_scale=s, v_scale=s)
    start = np.zeros(B, int)
    zero = np.zeros(tuple(pools[0].shape), np.uint8)
    for pool, rows in zip(pools, (new, -new)):
        want = fp4.append(zero, page, d, f64(rows), np.arange(0, B * n + 1, n), start, np.arange(B)[:, None], S)
        np.testing.assert_array_equal(pool.cpu().numpy(), want)
