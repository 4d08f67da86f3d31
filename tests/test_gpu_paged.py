"""GPU parity of the paged cache's attention and of the rows written into it, against the
float64 oracle, at the lengths, layouts and contents where they can go wrong."""
import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged
from paged_util import DEV, Cache, check_decode, f64, run_decode

pytestmark = pytest.mark.gpu

EDGE_LENS = [0, 1, 15, 16, 17, 63, 64, 65, 129, 0, 256, 300]


def ok():
    torch.cuda.synchronize()
    st = q.get_device_error()
    assert st == q.QUAIL_OK, q.status_string(st)


def queries(B, hq, d, seed=1, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(B, hq, d, generator=gen) * scale).bfloat16().to(DEV)


# ------------------------------------------------------------------ decode attention
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (8, 4), (4, 1), (16, 2), (32, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_lengths_and_heads(hq, hkv, d, fp8):
    cache = Cache(EDGE_LENS, hkv, d, 16, fp8, seed=hq + d)
    qt = queries(len(EDGE_LENS), hq, d)
    out, lse, score = run_decode(cache, qt, hq, scored=True)
    ok()
    check_decode(cache, qt, hq, out, lse, score)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_page_sizes(page, fp8):
    lens = [1, page - 1, page, page + 1, 5 * page + 3, 700]
    cache = Cache(lens, 2, 128, page, fp8, seed=page)
    qt = queries(len(lens), 8, 128)
    out, lse, _ = run_decode(cache, qt, 8)
    ok()
    check_decode(cache, qt, 8, out, lse)


@pytest.mark.parametrize("lens", [[40000], [20000, 1, 0, 9000], [33] * 700, [0, 0, 0], [0],
                                  [1] * 3, list(range(0, 900, 7))])
@pytest.mark.parametrize("d,fp8", [(128, False), (64, True)])
def test_splits(lens, d, fp8):
    """One sequence over many CTAs, many in one CTA, and both at once; with weights."""
    cache = Cache(lens, 2, d, 64, fp8, seed=len(lens))
    qt = queries(len(lens), 8, d)
    score_in = torch.rand(len(lens), 2, max(max(lens), 1) + 5, device=DEV)
    out, lse, score = run_decode(cache, qt, 8, scored=True, score_in=score_in)
    ok()
    check_decode(cache, qt, 8, out, lse, score, score_in)


@pytest.mark.parametrize("hq,hkv,B", [(2, 2, 320), (8, 4, 170), (4, 1, 640), (32, 4, 165), (16, 1, 700)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scored", [False, True])
def test_many_short_sequences(hq, hkv, B, d, fp8, scored):
    """At least 640 (sequence, head)s of at most 512 tokens: runs of warps."""
    rng = np.random.default_rng(hq + d)
    lens = rng.integers(0, 120, B).tolist()
    for b, n in ((0, 1), (1, 512), (2, 0), (5, 400), (B // 2, 257), (B - 2, 64), (B - 1, 499)):
        lens[b] = n
    cache = Cache(lens, hkv, d, 16 if d == 64 else 64, fp8, seed=hq)
    qt = queries(B, hq, d, seed=d)
    base = torch.rand(B, hkv, 512 + 5, device=DEV) if scored else None
    out, lse, score = run_decode(cache, qt, hq, scored, base)
    ok()
    some = {0, 1, 2, 3, 4, 5, B // 2, B - 2, B - 1} | set(rng.integers(0, B, 25).tolist())
    check_decode(cache, qt, hq, out, lse, score, base, only=some)
    again = run_decode(cache, qt, hq, scored, base)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    # a larger bound on the lengths takes the CTAs' runs; each within the bound of the true value
    wide = Cache(lens, hkv, d, cache.page, fp8, seed=hq, width=-(-2049 // cache.page))
    other = run_decode(wide, qt, hq, max_len=2049)
    ok()
    assert torch.allclose(out.float(), other[0].float(), rtol=2 ** -6, atol=2 ** -7)
    assert torch.allclose(lse, other[1], rtol=0, atol=1e-4)


def test_many_short_sequences_with_bad_pages_and_lengths():
    lens = [50] * 700
    cache = Cache(lens, 1, 64, 16, False)
    table = cache.table_np.copy()
    table[10, 1], table[699, 3], table[300, 0] = cache.pages, -1, 1 << 30
    cache.table = torch.from_numpy(table).to(DEV)
    n = torch.tensor(lens, dtype=torch.int32)
    n[20], n[400] = -1, 51
    cache.seq_lens = n.to(DEV)
    qt = queries(700, 4, 64)
    out, lse, score = run_decode(cache, qt, 4, True)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    bad = [10, 20, 300, 400, 699]
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    assert (score[[20, 400]] == -3.0).all() and (score[[10, 300, 699], :, :50] == 0).all()
    check_decode(cache, qt, 4, out, lse, score, only=[0, 9, 11, 19, 21, 299, 301, 399, 401, 698])


def test_weights_into_their_own_buffer_and_repeatable():
    cache = Cache([500, 31, 0, 3000], 2, 128, 32, False)
    qt = queries(4, 8, 128)
    start = torch.rand(4, 2, 3005, device=DEV)
    start[:, :, 3000:] = -3.0
    runs = []
    for _ in range(3):
        buf = start.clone()
        out, lse, _ = run_decode(cache, qt, 8, scored=True, score_in=buf, score_out=buf)
        ok()
        runs.append((out, lse, buf))
    for b, n in enumerate(cache.lens):
        assert torch.equal(runs[0][2][b, :, n:], start[b, :, n:])
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))
    other, _, score = run_decode(cache, qt, 8, scored=True, score_in=start)
    ok()
    assert torch.equal(other, runs[0][0])
    for b, n in enumerate(cache.lens):
        assert torch.equal(score[b, :, :n], runs[0][2][b, :, :n])


def test_row_strides_and_scale():
    """q as columns of a wider row, a scale of the caller's, max_seq_len above every length."""
    cache = Cache([70, 5, 260], 2, 64, 16, False, width=40)
    wide = queries(3, 12, 64).reshape(3, 12 * 64)
    qt = wide[:, 2 * 64:10 * 64].view(3, 8, 64)
    assert not qt.is_contiguous()
    out, lse, score = run_decode(cache, qt, 8, scored=True, max_len=640, scale=0.3)
    ok()
    check_decode(cache, qt, 8, out, lse, score, scale=0.3)


@pytest.mark.parametrize("fp8", [False, True])
def test_large_and_small_queries(fp8):
    """Scores far apart, far below and far above 1, and queries near the ends of bf16."""
    for scale in (1e-30, 1e-3, 12.0):
        cache = Cache([200, 1500], 1, 128, 16, fp8, seed=3)
        qt = queries(2, 4, 128, scale=scale)
        out, lse, score = run_decode(cache, qt, 4, scored=True)
        ok()
        check_decode(cache, qt, 4, out, lse, score)


def test_a_row_of_minus_infinity_keys():
    """Keys that give -inf take no weight; where all do, the sum is empty (NaN, -inf)."""
    cache = Cache([200, 40], 1, 64, 16, False)
    flat = cache.k.view(-1, 1, 64)
    qt = queries(2, 1, 64).abs()
    hidden = torch.from_numpy(paged.slots(cache.table_np[0], np.arange(64, 200), 16)).to(DEV)
    flat[hidden] = -float("inf")
    flat[torch.from_numpy(paged.slots(cache.table_np[1], np.arange(40), 16)).to(DEV)] = -float("inf")
    out, lse, _ = run_decode(cache, qt, 1)
    ok()
    cache.lens[0] = 64
    check_decode(cache, qt, 1, out, lse, only=[0])
    assert torch.isnan(out[1]).all() and (lse[1] == -float("inf")).all()


def test_shared_pages():
    """Two sequences that share a prefix's pages."""
    cache = Cache([100, 100], 2, 128, 16, False)
    cache.table_np[1, :4] = cache.table_np[0, :4]
    cache.table.copy_(torch.from_numpy(cache.table_np))
    qt = queries(2, 8, 128)
    out, lse, score = run_decode(cache, qt, 8, scored=True)
    ok()
    check_decode(cache, qt, 8, out, lse, score)


def test_a_contiguous_tensor_is_a_pool():
    T, hkv, d = 300, 2, 128
    k, v = (torch.randn(320, hkv, d, device=DEV).bfloat16() for _ in range(2))
    qt = queries(1, 8, d)
    table = torch.arange(20, dtype=torch.int32, device=DEV)[None]
    desc = q.make_paged_desc(1, T, 20, 16, 20, 8, hkv, d)
    out = torch.empty(1, 8, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    q.paged_decode_attn(desc, qt, k.view(20, 16, hkv, d), v.view(20, 16, hkv, d), table,
                        torch.tensor([T], dtype=torch.int32, device=DEV), out, ws)
    ok()
    ref, _, _ = paged.decode(f64(qt)[0], f64(k)[:T], f64(v)[:T], 1 / np.sqrt(d))
    assert np.abs(f64(out)[0] - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 1e-4


def test_pool_past_32_bits():
    """Pages whose element offsets exceed 2^31, and byte offsets 2^32."""
    hkv, d, page = 8, 128, 256
    pages = (1 << 32) // (page * hkv * d) + 64                # 2^32 values, 8.6 GB a pool
    lens = [700, 300]
    small = Cache(lens, hkv, d, page, False)
    k = torch.empty(pages, page, hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    shift = pages - small.pages
    k[shift:], v[shift:] = small.k, small.v
    small.k, small.v, small.pages = k, v, pages
    small.table = torch.where(small.table >= 0, small.table + shift, small.table)
    qt = queries(2, 32, d)
    out, lse, _ = run_decode(small, qt, 32)
    ok()
    small.lens = lens
    check_decode(small, qt, 32, out, lse)
    # and a new row at the far end of it
    desc = small.desc(32)
    new = torch.randn(2, hkv, d, device=DEV).bfloat16()
    pos = small.seq_lens - 1
    q.paged_kv_append(desc, new, new, pos, small.table, k, v)
    ok()
    for b in range(2):
        p = lens[b] - 1
        page_id = int(small.table[b, p // page])
        assert torch.equal(k[page_id, p % page], new[b]) and torch.equal(v[page_id, p % page], new[b])


def test_bad_pages_and_lengths_are_reported():
    """What is named outside the pool is not read: NaN for that sequence, the others right."""
    lens = [100, 200, 90, 0, 1500, 60]
    cache = Cache(lens, 2, 128, 16, False)
    qt = queries(len(lens), 8, 128)
    for bad in (-1, cache.pages, 1 << 30):
        table = cache.table_np.copy()
        table[1, 5] = bad
        table[4, 70] = bad
        cache.table = torch.from_numpy(table).to(DEV)
        out, lse, score = run_decode(cache, qt, 8, scored=True)
        torch.cuda.synchronize()
        assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
        assert q.get_device_error() == q.QUAIL_OK
        for b in (1, 4):
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
            assert (score[b, :, :lens[b]] == 0).all()
        check_decode(cache, qt, 8, out, lse, score, only=[0, 2, 3, 5])
    cache.table = torch.from_numpy(cache.table_np).to(DEV)
    cache.seq_lens = torch.tensor([100, -1, 90, 0, 1500, 1 << 30], dtype=torch.int32, device=DEV)
    out, lse, score = run_decode(cache, qt, 8, scored=True)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    for b in (1, 5):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
        assert (score[b] == -3.0).all()
    check_decode(cache, qt, 8, out, lse, score, only=[0, 2, 3, 4])


def test_other_stream_and_captured_graph():
    """Captured once, replayed after the lengths, pages and queries changed in place."""
    cache = Cache([900, 130, 40], 2, 128, 16, False, width=80)
    qt = queries(3, 8, 128)
    desc = cache.desc(8, max_len=1200)
    ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, 8, device=DEV)
    score = torch.full((3, 2, 1205), -3.0, device=DEV)

    def call(stream=None):
        q.paged_decode_attn(desc, qt, cache.k, cache.v, cache.table, cache.seq_lens, out, ws,
                            lse=lse, score_out=score, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    ok()
    check_decode(cache, qt, 8, out, lse, score)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    cache.lens = [5, 129, 0]
    cache.seq_lens.copy_(torch.tensor(cache.lens, dtype=torch.int32))
    qt.copy_(queries(3, 8, 128, seed=9))
    for _ in range(2):
        score.fill_(-3.0)
        out.fill_(1.0)
        graph.replay()
        ok()
        check_decode(cache, qt, 8, out, lse, score)


def test_binding_rejects_what_would_be_misread():
    cache = Cache([40, 20], 2, 64, 16, False)
    desc, qt = cache.desc(4), queries(2, 4, 64)
    ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
    good = dict(q=qt, k_pages=cache.k, v_pages=cache.v, block_table=cache.table,
                seq_lens=cache.seq_lens, out=torch.empty_like(qt), workspace=ws,
                lse=torch.empty(2, 4, device=DEV), score_out=torch.empty(2, 2, 40, device=DEV))
    q.paged_decode_attn(desc, **good)
    ok()
    for name, bad in [
            ("q", qt.half()), ("q", qt[:, :2]), ("q", qt.transpose(0, 1)), ("q", qt.cpu()),
            ("q", torch.empty(2, 4, 128, dtype=torch.bfloat16, device=DEV)[:, :, ::2]),
            ("k_pages", cache.k[:, :8]), ("v_pages", cache.v.float()),
            ("k_pages", cache.k.view(torch.uint8)[..., :64]), ("v_pages", cache.v.transpose(1, 2)),
            ("block_table", cache.table.long()), ("block_table", cache.table[:, :-1]),
            ("seq_lens", cache.seq_lens.long()), ("seq_lens", cache.seq_lens[:1]),
            ("seq_lens", cache.seq_lens.cpu()), ("out", torch.empty(2, 4, 64, device=DEV)),
            ("out", torch.empty(2, 64, 4, dtype=torch.bfloat16, device=DEV).transpose(1, 2)),
            ("workspace", ws.float()), ("lse", torch.empty(4, 2, device=DEV)),
            ("score_out", torch.empty(2, 2, 39, device=DEV)),
            ("score_out", torch.empty(2, 2, 40, device=DEV, dtype=torch.bfloat16))]:
        with pytest.raises(ValueError, match=name):
            q.paged_decode_attn(desc, **{**good, name: bad})
    with pytest.raises(ValueError, match="score_in"):
        q.paged_decode_attn(desc, **{**good, "score_out": None}, score_in=good["score_out"])
    with pytest.raises(q.QuailError, match="INVALID_ARG"):
        q.paged_decode_attn(desc, **{**good, "workspace": ws[:64]})
    with pytest.raises(ValueError, match="scale"):
        q.paged_decode_attn(desc, **good, k_scale=torch.ones(2, 2, device=DEV))
    ok()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (8, 128, 64), (2, 128, 256), (3, 64, 32)])
def test_append_prompts_and_tokens(hkv, d, page, fp8):
    rng = np.random.default_rng(d + page)
    counts = [0, 1, 5, 33, 0, 130, 2]
    start = [7, page, 0, page - 1, 3, 2 * page - 5, 0]
    ends = [s + c for s, c in zip(start, counts)]
    table, pages = __import__("paged_util").block_table(ends, page, rng)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k = torch.randint(0, 100, (pages, page, hkv, d), dtype=torch.uint8)
    k = k.view(dt) if fp8 else k.to(dt)
    v = k.clone()
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    row = torch.randn(off[-1], (2 * hkv + 1) * d).bfloat16()
    row[0, :8] = torch.tensor([0.0, -0.0, 1e30, -1e30, 3e38, 1e-38, float("inf"), -float("inf")])
    new = [row[:, d:(hkv + 1) * d].view(-1, hkv, d), row[:, (hkv + 1) * d:].view(-1, hkv, d)]
    scales = [torch.rand(len(counts), hkv) * 0.02 + 1e-3 for _ in range(2)] if fp8 else [None] * 2
    if fp8:  # scales at the ends of fp32, where the quotient must be divided
        scales[0][2, 0], scales[1][2, 0] = 1e-25, 1e25
        scales[0][3, 0], scales[1][3, 0] = 1e-40, 3e38
    desc = q.make_paged_desc(len(counts), max(ends), pages, page, table.shape[1], 2 * hkv, hkv, d,
                             kv_fp8=fp8)
    gpu = row.to(DEV)
    gk, gv = k.to(DEV), v.to(DEV)
    q.paged_kv_append(desc, gpu[:, d:(hkv + 1) * d].view(-1, hkv, d),
                      gpu[:, (hkv + 1) * d:].view(-1, hkv, d),
                      torch.tensor(start, dtype=torch.int32, device=DEV),
                      torch.from_numpy(table).to(DEV), gk, gv,
                      new_offsets=torch.from_numpy(off).to(DEV),
                      k_scale=None if not fp8 else scales[0].to(DEV),
                      v_scale=None if not fp8 else scales[1].to(DEV))
    ok()
    for before, rows, s, got in ((k, new[0], scales[0], gk), (v, new[1], scales[1], gv)):
        raw = torch.uint8 if fp8 else torch.int16
        pages_np = before.view(raw).numpy()
        rows_np = rows.contiguous().float().numpy() if fp8 else rows.contiguous().view(raw).numpy()
        want = paged.append(pages_np, rows_np, off, start, table,
                            None if s is None else s.numpy())
        np.testing.assert_array_equal(got.view(raw).cpu().numpy(), want.astype(pages_np.dtype))
    # one token each, without offsets
    one = torch.randn(len(counts), hkv, d).bfloat16()
    pos = [max(e - 1, 0) for e in ends]
    q.paged_kv_append(desc, one.to(DEV), one.to(DEV),
                      torch.tensor(pos, dtype=torch.int32, device=DEV),
                      torch.from_numpy(table).to(DEV), gk, gv,
                      k_scale=None if not fp8 else scales[0].to(DEV),
                      v_scale=None if not fp8 else scales[1].to(DEV))
    ok()
    rows_np = one.float().numpy() if fp8 else one.view(torch.int16).numpy()
    raw = torch.uint8 if fp8 else torch.int16
    base = np.arange(len(counts) + 1)
    k1 = paged.append(k.view(raw).numpy(), (new[0].contiguous().float() if fp8 else new[0].contiguous().view(raw)).numpy(),
                      off, start, table, None if not fp8 else scales[0].numpy())
    k2 = paged.append(k1, rows_np, base, pos, table, None if not fp8 else scales[0].numpy())
    np.testing.assert_array_equal(gk.view(raw).cpu().numpy(), k2.astype(k1.dtype))


def test_append_codes_are_the_quantisers():
    """The codes that quail_quantize_kv_fp8 gives for the same tensor and scales."""
    T, hkv, d = 512, 2, 128
    x = torch.randn(T, hkv, d, device=DEV).bfloat16()
    codes = torch.empty(T, hkv, d, dtype=torch.uint8, device=DEV)
    scale = torch.empty(1, hkv, device=DEV)
    q.quantize_kv_fp8(x, torch.tensor([0, T], dtype=torch.int32, device=DEV), codes, scale)
    pages = torch.zeros(T // 16, 16, hkv, d, dtype=torch.uint8, device=DEV)
    other = torch.zeros_like(pages)
    table = torch.arange(T // 16, dtype=torch.int32, device=DEV)[None]
    desc = q.make_paged_desc(1, T, T // 16, 16, T // 16, 4, hkv, d, kv_fp8=True)
    q.paged_kv_append(desc, x, x, torch.zeros(1, dtype=torch.int32, device=DEV), table, pages, other,
                      new_offsets=torch.tensor([0, T], dtype=torch.int32, device=DEV),
                      k_scale=scale, v_scale=scale)
    ok()
    assert torch.equal(pages.view(T, hkv, d), codes) and torch.equal(other, pages)


def test_append_skips_and_reports_what_is_out_of_range():
    hkv, d, page = 2, 64, 16
    k = torch.zeros(4, page, hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    new = torch.ones(4, hkv, d, dtype=torch.bfloat16, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    desc = q.make_paged_desc(4, 30, 4, page, 2, 4, hkv, d)
    table = i32([[0, 1], [-1, 4], [2, 9], [3, 3]])
    for start, written in (([0, 3, 20, -1], {(0, 0)}), ([29, 0, 30, 2 ** 31 - 1], {(1, 13)}),
                           ([5, 17, 1, 31], {(0, 5), (2, 1)})):
        k.zero_(), v.zero_()
        q.paged_kv_append(desc, new, new, i32(start), table, k, v)
        torch.cuda.synchronize()
        assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
        got = {tuple(x) for x in (k != 0).any(-1).any(-1).nonzero().tolist()}
        assert got == written and torch.equal(k, v)
    # offsets that do not agree with the rows: those that no sequence holds are skipped
    for off, written in (([0, 1, 1, 1, 3], {(0, 0), (3, 0), (3, 1)}), ([1, 2, 2, 2, 4], {(0, 0), (3, 0), (3, 1)}),
                         ([0, 3, 2, 2, 4], None), ([0, 9, 9, 9, 9], None)):
        k.zero_(), v.zero_()
        q.paged_kv_append(desc, new, new, i32([0, 0, 0, 0]), table, k, v, new_offsets=i32(off))
        torch.cuda.synchronize()
        assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
        if written is not None:
            got = {tuple(x) for x in (k != 0).any(-1).any(-1).nonzero().tolist()}
            assert got == written
