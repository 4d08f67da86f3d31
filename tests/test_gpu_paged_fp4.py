"""GPU tests of 4-bit pages against the oracle: rows quantised as they are appended (bit for bit),
rows read back (to a rounding), single-token attention with the weights that tokens receive, the
operators one after the other, and what bad arguments leave behind."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import fp4, paged
from paged_fp4_util import Cache4, check_decode, queries, run_decode
from paged_util import BF16, DEV, U32, block_table, f64

pytestmark = pytest.mark.gpu
DEVICE_BOUNDS = q.QUAIL_ERR_DEVICE_BOUNDS


@pytest.fixture(autouse=True)
def no_device_error():
    q.get_device_error()
    yield
    assert q.get_device_error() == q.QUAIL_OK


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Rows:
    """New rows for sequences, empty pages with a pattern in them, and the call's arguments."""

    def __init__(self, counts, start, hkv, d, page, seed=0, pad=0, scale=None):
        rng = np.random.default_rng(seed)
        self.counts, self.start, self.hkv, self.d, self.page = counts, start, hkv, d, page
        T, B = int(sum(counts)), len(counts)
        self.off_np = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.table_np, self.pages = block_table(np.add(counts, start), page, rng)
        x = torch.from_numpy(rng.normal(size=(2, T, hkv * d + pad)).astype(np.float32)).bfloat16()
        self.x = x.to(DEV)
        self.k_new, self.v_new = (self.x[i, :, pad:].view(T, hkv, d) if not pad else
                                  self.x[i].as_strided((T, hkv, d), (hkv * d + pad, d, 1), self.x[i].storage_offset() + pad)
                                  for i in range(2))
        amax = np.abs(x[:, :, pad:].float().numpy()).max() if T else 1.0
        self.ks_np, self.vs_np = ((np.float32(amax) / 2688 * (0.4 + rng.random((B, hkv)))).astype(np.float32)
                                  if scale is None else np.full((B, hkv), scale, np.float32)
                                  for _ in range(2))
        self.pool_np = rng.integers(0, 256, (self.pages, hkv, page * d * 9 // 16), dtype=np.uint8)
        self.k, self.v = (torch.from_numpy(self.pool_np).to(DEV) for _ in range(2))
        self.desc = q.make_paged_desc(B, int(max(np.add(counts, start), default=0)), self.pages, page,
                                      self.table_np.shape[1], hkv, hkv, d, kv_fp4=True)
        self.kw = dict(k_scale=torch.from_numpy(self.ks_np).to(DEV), v_scale=torch.from_numpy(self.vs_np).to(DEV))
        self.table, self.start_t, self.off = i32(self.table_np), i32(start), i32(self.off_np)

    def append(self, off=True, **kw):
        q.paged_kv_append(self.desc, self.k_new, self.v_new, self.start_t, self.table, self.k, self.v,
                          new_offsets=self.off if off else None, **{**self.kw, **kw})

    def want(self):
        return [fp4.append(self.pool_np, self.page, self.d, f64(x), self.off_np, self.start, self.table_np, s)
                for x, s in ((self.k_new, self.ks_np), (self.v_new, self.vs_np))]


ROWS = [
    ([1], [0], 1, 64, 16, 0), ([1, 1, 1], [5, 0, 31], 8, 128, 16, 0), ([3], [14], 2, 64, 16, 64),
    ([65, 0, 130], [0, 7, 63], 4, 128, 64, 256), ([1000], [17], 3, 128, 256, 0),
    ([17, 64, 1, 33], [0, 0, 100, 15], 16, 64, 32, 8), ([700, 3, 901], [5, 1, 0], 8, 128, 128, 0),
]


@pytest.mark.parametrize("counts,start,hkv,d,page,pad", ROWS)
def test_append_bit_for_bit_and_read(counts, start, hkv, d, page, pad):
    r = Rows(counts, start, hkv, d, page, seed=len(counts), pad=pad)
    r.append(off=counts != [1, 1, 1])
    want = r.want()
    np.testing.assert_array_equal(r.k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(r.v.cpu().numpy(), want[1])
    # back again, into columns of wider rows
    T = int(sum(counts))
    wide = torch.full((T, 2 * hkv * d + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out, v_out = (wide.as_strided((T, hkv, d), (wide.shape[1], d, 1), o) for o in (8, 8 + hkv * d))
    q.paged_kv_read(r.desc, r.k, r.v, r.start_t, r.table, k_out, v_out, offsets=r.off, **r.kw)
    for got, pool, s in ((k_out, want[0], r.ks_np), (v_out, want[1], r.vs_np)):
        got = f64(got)
        for b in range(len(counts)):
            ref = fp4.rows(pool, page, d, r.table_np[b], start[b] + np.arange(counts[b]), s[b])
            ref = torch.from_numpy(ref.astype(np.float32)).bfloat16()    # the product in fp32, then bf16
            np.testing.assert_array_equal(got[r.off_np[b]:r.off_np[b + 1]], f64(ref))
    assert (f64(wide)[:, :8] == 7).all() and (f64(wide)[:, 8 + 2 * hkv * d:] == 7).all()


@pytest.mark.parametrize("scale", [1.0, 0.01, 2.0 ** -100, 2.0 ** 100, -0.003, 3e38, 1e-45, 0.0, math.inf, math.nan])
def test_append_scales(scale):
    """Scales of every size: quotients past fp32, below it, and none."""
    r = Rows([40], [0], 2, 128, 16, seed=3, scale=scale)
    r.append()
    want = r.want()
    np.testing.assert_array_equal(r.k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(r.v.cpu().numpy(), want[1])


def test_append_every_tie():
    """Quotients on and next to the borders between codes, and of block scales."""
    grid = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7])
    near = np.concatenate([grid * (1 + e) for e in (-2.0 ** -7, 0, 2.0 ** -7)])
    r = Rows([1024], [0], 2, 64, 16, seed=4, scale=2.0 ** -7)
    rng = np.random.default_rng(4)
    x = rng.choice(near, (1024, 2, 64)) * rng.choice([-1, 1], (1024, 2, 64)) * 2.0 ** rng.integers(-9, 6, (1024, 2, 1))
    # the block's largest decides its scale: 6 b S for scales b of four bits, and borders between them
    x[:, :, ::16] = 6 * (rng.integers(16, 33, (1024, 2, 4)) / 16) * 2.0 ** rng.integers(-8, 7, (1024, 2, 1))
    r.x.copy_(torch.from_numpy(np.stack([x, -x]).reshape(2, 1024, -1)).bfloat16())
    r.append()
    want = r.want()
    np.testing.assert_array_equal(r.k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(r.v.cpu().numpy(), want[1])


def test_append_specials():
    """NaN makes its block NaN, infinities saturate, zeros and what is far below the scale are zeros."""
    r = Rows([64], [0], 2, 64, 16, seed=5)
    x = r.x.view(2, 64, 2, 64)
    x[:, 0, 0, 5], x[:, 1, 1, 63] = math.nan, -math.nan
    x[:, 2, 0, 16:32], x[:, 3, 1, 0] = math.inf, -math.inf
    x[:, 4], x[:, 5], x[:, 6] = 0.0, -0.0, 1e-30
    x[:, 7, 0], x[:, 8] = 3.3e38, 1e-40
    r.append()
    want = r.want()
    np.testing.assert_array_equal(r.k.cpu().numpy(), want[0])
    np.testing.assert_array_equal(r.v.cpu().numpy(), want[1])


@pytest.mark.parametrize("form", ["bf16", "fp8"])
@pytest.mark.parametrize("hkv,d,page", [(8, 128, 16), (3, 64, 64)])
def test_read_of_the_other_forms(form, hkv, d, page):
    lens, start = [70, 1, 0, 300], [3, 0, 0, 129]
    rng = np.random.default_rng(7)
    table_np, pages = block_table(np.add(lens, start), page, rng)
    x = torch.randn(2, pages, page, hkv, d, generator=torch.Generator().manual_seed(7))
    x = (x * 90).clamp(-448, 448).to(torch.float8_e4m3fn) if form == "fp8" else x.bfloat16()
    x = x.to(DEV)
    scale = (torch.rand(2, 4, hkv, generator=torch.Generator().manual_seed(8)) / 90).to(DEV)
    kw = dict(k_scale=scale[0], v_scale=scale[1]) if form == "fp8" else {}
    desc = q.make_paged_desc(4, 430, pages, page, max(table_np.shape[1], -(-430 // page)), hkv, hkv, d,
                             kv_fp8=form == "fp8")
    table = np.full((4, desc.max_pages_per_seq), -1, np.int32)
    table[:, :table_np.shape[1]] = table_np
    off = np.concatenate([[0], np.cumsum(lens)])
    outs = [torch.zeros(off[-1], hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q.paged_kv_read(desc, x[0], x[1], i32(start), i32(table), *outs, offsets=i32(off), **kw)
    for i, got in enumerate(outs):
        flat = x[i].float().view(-1, hkv, d).cpu()
        for b in range(4):
            at = paged.slots(table[b], start[b] + np.arange(lens[b]), page)
            ref = flat[at] * (scale[i, b].cpu()[None, :, None] if form == "fp8" else 1.0)
            np.testing.assert_array_equal(f64(got[off[b]:off[b + 1]]), f64(ref.bfloat16()))


def test_read_one_side_and_single_rows():
    c = Cache4([30, 5, 70], 2, 128, 16, seed=1)
    desc = c.desc(2, 80)
    desc = q.make_paged_desc(3, 70, c.pages, 16, c.table.shape[1], 2, 2, 128, kv_fp4=True)
    out = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=DEV)
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    for side, (k_out, v_out) in enumerate(((out, None), (None, out))):
        out.fill_(9)
        q.paged_kv_read(desc, None if side else c.k, c.v if side else None, i32([29, 0, 40]), c.table, k_out,
                        v_out, **kw)
        for b, at in enumerate((29, 0, 40)):
            ref = c.rows(b, [at])[side][0].astype(np.float32)
            np.testing.assert_array_equal(f64(out[b]), f64(torch.from_numpy(ref).bfloat16()))


def test_rows_that_name_nothing():
    """Bad positions, pages and offsets: reported; append leaves the pages, read gives NaN, or leaves
    rows that no sequence holds."""
    r = Rows([4, 4, 4], [0, 0, 60], 2, 64, 16, seed=6)
    table = r.table_np.copy()
    table[1, 0] = r.pages
    start = i32([-1, 0, 62])                       # below zero; a bad page; past max_seq_len from row 2 on
    q.paged_kv_append(r.desc, r.k_new, r.v_new, start, i32(table), r.k, r.v, new_offsets=r.off, **r.kw)
    assert q.get_device_error() == DEVICE_BOUNDS
    want = fp4.append(r.pool_np, 16, 64, f64(r.k_new)[8:10], [0, 2], [62], table[2:], r.ks_np[2:])
    np.testing.assert_array_equal(r.k.cpu().numpy(), want)
    outs = [torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    q.paged_kv_read(r.desc, r.k, r.v, start, i32(table), *outs, offsets=r.off, **r.kw)
    assert q.get_device_error() == DEVICE_BOUNDS
    for x in outs:
        x = f64(x)
        assert np.isnan(x[:8]).all() and np.isfinite(x[8:10]).all() and np.isnan(x[10:]).all()
    # offsets that leave rows to nobody
    outs = [torch.full((12, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    before = r.k.clone()
    q.paged_kv_read(r.desc, r.k, r.v, r.start_t, r.table, *outs, offsets=i32([2, 4, 8, 9]), **r.kw)
    assert q.get_device_error() == DEVICE_BOUNDS
    x = f64(outs[0])
    assert (x[:2] == 5).all() and (x[9:] == 5).all() and (x[2:9] != 5).any(axis=(1, 2)).all()
    q.paged_kv_append(r.desc, r.k_new, r.v_new, r.start_t, r.table, r.k, r.v, new_offsets=i32([12, 12, 12, 12]),
                      **r.kw)
    assert q.get_device_error() == DEVICE_BOUNDS
    assert torch.equal(before, r.k)


def test_empty_calls():
    d0 = q.make_paged_desc(0, 0, 4, 16, 0, 4, 2, 64, kv_fp4=True)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)
    pool, kw = z(4, 2, 16 * 36, t=torch.uint8), dict(k_scale=z(0, 2, t=torch.float32), v_scale=z(0, 2, t=torch.float32))
    none, table = z(0, t=torch.int32), z(0, 0, t=torch.int32)
    q.paged_kv_append(d0, z(0, 2, 64), z(0, 2, 64), none, table, pool, pool.clone(), **kw)
    q.paged_kv_read(d0, pool, pool.clone(), none, table, z(0, 2, 64), z(0, 2, 64), **kw)
    ws = z(q.paged_decode_workspace_size(d0) + 16, t=torch.uint8)
    q.paged_decode_attn(d0, z(0, 4, 64), pool, pool.clone(), table, none, z(0, 4, 64), ws, **kw)
    r = Rows([0, 0], [3, 0], 2, 64, 16)
    r.append()
    np.testing.assert_array_equal(r.k.cpu().numpy(), r.pool_np)


DECODE = [
    # lens, hq, hkv, d, page: one cluster, whole batch, runs of warps, one long, every group
    ([1], 1, 1, 64, 16), ([1, 2, 31, 32, 33], 8, 2, 128, 16), ([777], 32, 8, 128, 16),
    ([127, 128, 129, 0, 15, 16, 17], 16, 1, 128, 32), ([300, 5, 0, 64], 4, 4, 64, 256),
    ([2000, 900, 3000], 32, 8, 128, 64), ([5000], 6, 3, 64, 128), ([4000, 4001, 100], 48, 3, 128, 16),
    ([20 + i % 64 for i in range(181)], 64, 4, 128, 16), ([1 + i % 100 for i in range(170)], 32, 4, 64, 32),
    ([600, 20, 900, 3] * 60, 8, 4, 128, 16), ([30011], 16, 2, 128, 256), ([20000, 3], 32, 2, 64, 64),
]


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("lens,hq,hkv,d,page", DECODE)
def test_decode(lens, hq, hkv, d, page, scored):
    c = Cache4(lens, hkv, d, page, seed=hq + len(lens))
    qt = queries(5, len(lens), hq, d, scale=1.5)
    score_in = None
    if scored:
        score_in = torch.rand(len(lens), hkv, max(lens) + 5, device=DEV)
    out, lse, score = run_decode(c, qt, hq, scored, score_in)
    check_decode(c, qt, hq, out, lse, score, score_in,
                 only=None if len(lens) < 50 else set(range(0, len(lens), 7)))


@pytest.mark.parametrize("blocks", [(0x01, 0x7E), (0x00, 0x07), (0x7E, 0x7E), (0x81, 0xFE)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_block_scales_of_every_size(blocks, d):
    """The whole range of e4m3, its subnormals, its largest, negative ones."""
    c = Cache4([333, 40], 2, d, 16, seed=2, blocks=blocks)
    qt = queries(2, 2, 8, d, scale=0.3)
    check_decode(c, qt, 8, *run_decode(c, qt, 8)[:2])


@pytest.mark.parametrize("scale", [0.0, 0.7, 1e-3])
@pytest.mark.parametrize("size", [1e-30, 1.0, 1e4])
def test_decode_queries_of_every_size(scale, size):
    c = Cache4([200, 17], 2, 128, 32, seed=9)
    c.ks_np = (c.ks_np / np.float32(max(size, 1.0))).astype(np.float32)
    c.k_scale = torch.from_numpy(c.ks_np).to(DEV)
    qt = queries(3, 2, 4, 128, scale=size)
    check_decode(c, qt, 4, *run_decode(c, qt, 4, scale=scale)[:2], scale=scale)


def test_decode_strided_queries_and_bound_above_the_lengths():
    c = Cache4([60, 200, 7], 2, 128, 16, seed=4, width=64)
    wide = queries(8, 3, 3 * 8 * 128)
    qt = wide.as_strided((3, 8, 128), (wide.shape[1], 128, 1), 64)
    for max_len in (200, 1024):
        out, lse, score = run_decode(c, qt, 8, True, max_len=max_len)
        check_decode(c, qt, 8, out, lse, score)


def test_decode_nan_blocks_and_bad_pages():
    """A block scale that is NaN gives NaN to the heads that see it, a bad page or length NaN and a
    report; other sequences and heads are as they would be."""
    c = Cache4([100, 100, 100, 100], 2, 128, 16, seed=11)
    qt = queries(11, 4, 8, 128)
    codes, blocks = fp4.parts(c.k_np, 16, 128)
    blocks = blocks.copy()
    blocks[c.table_np[1, 3], 1, 2, 4] = 0x7F
    k = torch.from_numpy(fp4.join(codes, blocks)).to(DEV)
    table, lens = c.table.clone(), c.seq_lens.clone()
    table[2, 6] = c.pages
    lens[3] = 101
    desc = c.desc(8, 100)
    out = torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(4, 8, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    q.paged_decode_attn(desc, qt, k, c.v, table, lens, out, ws, lse=lse, k_scale=c.k_scale, v_scale=c.v_scale)
    assert q.get_device_error() == DEVICE_BOUNDS
    o, l_ = f64(out), f64(lse)
    assert np.isnan(o[1, 4:]).all() and np.isnan(l_[1, 4:]).all() and np.isfinite(o[1, :4]).all()
    assert np.isnan(o[2:]).all() and np.isnan(l_[2:]).all()
    check_decode(c, qt, 8, out, lse, only={0})


def test_decode_does_not_depend_on_timing_or_what_lies_behind():
    c = Cache4([3000, 129, 640], 4, 128, 16, seed=12)
    qt = queries(12, 3, 16, 128)
    first = run_decode(c, qt, 16, True)
    for _ in range(3):
        again = run_decode(c, qt, 16, True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_prompts_tokens_attention_and_reading_back():
    """Prompts quantised into pages, tokens appended one at a time and attended to, the rows read
    back as anchors of a cascade over the same keys."""
    hq, hkv, d, page, lens, steps = 8, 2, 128, 16, [150, 40, 77], 20
    B, T, L = 3, sum(lens), max(lens) + steps
    x = [queries(20 + i, T, hkv, d) for i in range(2)]
    amax = [max(float(t.abs().max()), 4.5) for t in x]
    scale = [torch.full((B, hkv), a / 2688, device=DEV) for a in amax]
    width = -(-L // page)
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).view(B, width).int().to(DEV)
    desc = q.make_paged_desc(B, L, B * width, page, width, hq, hkv, d, kv_fp4=True)
    pools = [torch.zeros(q.paged_pool_shape(desc), dtype=torch.uint8, device=DEV) for _ in range(2)]
    kw = dict(k_scale=scale[0], v_scale=scale[1])
    off = i32(np.concatenate([[0], np.cumsum(lens)]))
    q.paged_kv_append(desc, *x, i32([0] * B), table, *pools, new_offsets=off, **kw)
    lens_t = i32(lens)
    ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
    score = torch.zeros(B, hkv, L, device=DEV)
    total = np.zeros((B, hkv, L))
    for step in range(steps):
        new = [queries(100 + 2 * step + i, B, hkv, d) for i in range(2)]
        qt = queries(300 + step, B, hq, d)
        q.paged_kv_append(desc, *new, lens_t, table, *pools, **kw)
        lens_t = lens_t + 1
        out = torch.empty(B, hq, d, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(B, hq, device=DEV)
        q.paged_decode_attn(desc, qt, *pools, table, lens_t, out, ws, lse=lse, score_in=score, score_out=score, **kw)
        for b in range(B):
            n = lens[b] + step + 1
            k, v = (fp4.rows(p.cpu().numpy(), page, d, table[b].cpu().numpy(), np.arange(n), f64(s)[b])
                    for p, s in zip(pools, scale))
            ref, ref_lse, w = paged.decode(f64(qt)[b], k, v, 1 / math.sqrt(d))
            total[b, :, :n] += w
            np.testing.assert_allclose(f64(out)[b], ref, atol=1e-5, rtol=2 * BF16)
            np.testing.assert_allclose(f64(lse)[b], ref_lse, atol=1e-5)
    np.testing.assert_allclose(f64(score), total, atol=1e-5, rtol=1e-4)
    # the cache as anchors: 2 suffixes of each sequence's rows read back
    n = np.array(lens) + steps
    A = int(n.sum())
    ka, va = (torch.empty(A, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ao = np.concatenate([[0], np.cumsum(n)])
    q.paged_kv_read(desc, *pools, i32([0] * B), table, ka, va, offsets=i32(ao), **kw)
    S = 6 * 10
    qs, ks, vs = queries(7, S, hq, d), queries(8, S, hkv, d), queries(9, S, hkv, d)
    cd = q.make_desc(B, 6, A, S, int(n.max()), 10, hq, hkv, d)
    cws = torch.empty(q.cascade_workspace_size(cd), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty(S, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(S, hq, device=DEV)
    q.cascade_attn(cd, qs, ka, va, ks, vs, i32(ao), i32([0, 2, 4, 6]), i32(range(0, 61, 10)), out, lse, cws)
    import oracle
    rows = [np.concatenate([fp4.rows(p.cpu().numpy(), page, d, table[b].cpu().numpy(), np.arange(n[b]), f64(s)[b])
                            for b in range(B)]) for p, s in zip(pools, scale)]
    ref, ref_lse = oracle.cascade_attention(f64(qs), *rows, f64(ks), f64(vs), ao, [0, 2, 4, 6],
                                            np.arange(0, 61, 10), 1 / math.sqrt(d))
    rel = np.linalg.norm(f64(out) - ref) / np.linalg.norm(ref)
    # the library's bound for the cascade, and a rounding of K (in the scores) and V to bf16
    assert rel <= 5e-3 + 2 * BF16 and np.abs(f64(lse) - ref_lse).max() <= 2e-2


def test_captured_and_replayed_with_new_inputs():
    c = Cache4([500, 20, 131], 2, 128, 16, seed=13, width=40)
    hq = 8
    desc = c.desc(hq, 600)
    qt, lens = queries(13, 3, hq, 128), c.seq_lens.clone()
    new = [queries(14 + i, 3, 2, 128) for i in range(2)]
    out, lse = torch.empty(3, hq, 128, dtype=torch.bfloat16, device=DEV), torch.empty(3, hq, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    k, v = c.k.clone(), c.v.clone()
    table = c.table.clone()
    # room for one token more in every sequence: a page of its own where the last one is full
    spare = iter(np.setdiff1d(np.arange(c.pages), c.table_np))
    for b, n in enumerate(c.lens):
        if n % 16 == 0:
            table[b, n // 16] = int(next(spare))
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    back = [torch.empty(3, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def step():
        q.paged_kv_append(desc, *new, lens, table, k, v, **kw)
        more = lens + 1
        q.paged_decode_attn(desc, qt, k, v, table, more, out, ws, lse=lse, **kw)
        q.paged_kv_read(desc, k, v, lens, table, *back, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (50, 60):
        for i in range(2):
            new[i].copy_(queries(seed + i, 3, 2, 128))
        qt.copy_(queries(seed + 5, 3, hq, 128))
        out.zero_()
        graph.replay()
        for b in range(3):
            n = c.lens[b] + 1
            rows = [fp4.rows(p.cpu().numpy(), 16, 128, table[b].cpu().numpy(), np.arange(n), s[b])
                    for p, s in ((k, c.ks_np), (v, c.vs_np))]
            ref, ref_lse, _ = paged.decode(f64(qt)[b], *rows, 1 / math.sqrt(128))
            np.testing.assert_allclose(f64(out)[b], ref, atol=1e-5, rtol=2 * BF16)
            np.testing.assert_allclose(f64(lse)[b], ref_lse, atol=2e-5)
            got = f64(back[0])[b]
            np.testing.assert_allclose(got, rows[0][-1], rtol=BF16 + 2 * U32)


def test_on_another_stream():
    c = Cache4([900, 33], 4, 64, 32, seed=15)
    qt = queries(15, 2, 8, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    desc = c.desc(8)
    out, lse = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 8, device=DEV)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    s.wait_stream(torch.cuda.current_stream())
    q.paged_decode_attn(desc, qt, c.k, c.v, c.table, c.seq_lens, out, ws, lse=lse, k_scale=c.k_scale,
                        v_scale=c.v_scale, stream=s)
    s.synchronize()
    check_decode(c, qt, 8, out, lse)
