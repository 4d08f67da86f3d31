"""Host-only checks of the calls on 4-bit pages: the C ABI refuses bad arguments before any
launch, and the binding refuses tensors that the library would misread."""
import ctypes

import pytest
import torch

import prefill_only_cascade_gb300 as q
from test_abi_paged import BAD_DESCS, BIG, INVALID, P, append, decode, desc

FP4 = dict(kv_fp4=True)


def read(d, **o):
    a = dict(num=4, off=None, start=P, table=P, ks=None, vs=None, kp=P, vp=P + (1 << 40), k=BIG,
             v=2 * BIG, ks_=1024, vs_=1024)
    a.update(o)
    return q.lib.quail_paged_kv_read(None if d is None else ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("change,expect", BAD_DESCS)
@pytest.mark.parametrize("form", [dict(), FP4])
def test_bad_descriptors(change, expect, form):
    d = desc(**change, **form)
    s = dict(ks=P, vs=P) if form else {}
    assert read(d, num=d.num_seqs, **s) == expect
    assert append(d, num_new=d.num_seqs, **s) == expect
    assert decode(d, **s) == expect
    assert q.paged_page_bytes(d) == 0


def test_null_descriptor_and_unknown_form():
    assert read(None) == INVALID
    assert q.lib.quail_paged_page_bytes(None) == 0
    d = desc()
    for form in (3, -1):
        d.kv_dtype = form
        assert read(d, ks=P, vs=P) == append(d, ks=P, vs=P) == decode(d, ks=P, vs=P) == INVALID


def test_page_bytes():
    assert q.paged_page_bytes(desc()) == 16 * 8 * 128 * 2
    assert q.paged_page_bytes(desc(kv_fp8=True)) == 16 * 8 * 128
    assert q.paged_page_bytes(desc(**FP4)) == 16 * 8 * (64 + 8)
    assert q.paged_page_bytes(desc(head_dim=64, page_size=256, **FP4)) == 256 * 8 * (32 + 4)
    d = desc(head_dim=64, page_size=256, **FP4)
    n, hkv, head = q.paged_pool_shape(d)
    assert (n, hkv * head) == (100, q.paged_page_bytes(d)) and q.paged_pool_shape(d, 7)[0] == 7
    assert q.paged_pool_shape(desc()) == (100, 16, 8, 128)


@pytest.mark.parametrize("change", [
    dict(num=-1), dict(num=5), dict(num=1 << 31, off=P), dict(start=None), dict(table=None),
    dict(start=P + 2), dict(table=P + 1), dict(off=P + 2), dict(k=None, v=None), dict(kp=None),
    dict(vp=None), dict(kp=P + 8), dict(vp=P + 4), dict(k=BIG + 8), dict(v=BIG + 2),
    dict(ks_=1023), dict(ks_=1028), dict(vs_=1000), dict(ks=P), dict(ks=P, vs=P),
    dict(v=BIG), dict(v=BIG + 512), dict(k=P), dict(k=P + (1 << 40)),   # outputs over each other, over pages
    dict(k=P - 4 * 2048 + 16, num=4), dict(v=P + 100 * 16 * 8 * 256 - 16),
])
def test_read_refuses(change):
    assert read(desc(), **change) == INVALID


def test_read_takes_columns_of_one_row():
    """K and V side by side in one wider row do not overlap; overlapping columns do."""
    assert read(desc(), k=BIG, v=BIG + 2048 - 16, ks_=2048, vs_=2048) == INVALID
    assert read(desc(), k=BIG, v=BIG + 2048 + 16, ks_=2048, vs_=2048) == INVALID
    assert read(desc(), k=BIG, v=BIG + 2048, ks_=2048, vs_=2048) != INVALID   # no device here, or done


def test_codes_need_scales():
    for d in (desc(kv_fp8=True), desc(**FP4)):
        for s in (dict(), dict(ks=P), dict(vs=P), dict(ks=P, vs=P + 2)):
            assert read(d, **s) == append(d, **s) == decode(d, **s) == INVALID


def test_fp4_pool_sizes_count_in_overlaps():
    """K and V pools that touch at their ends are told apart by the form's own page size."""
    d = desc(**FP4)
    pool = 100 * 16 * 8 * 72
    assert append(d, ks=P, vs=P, kp=BIG, vp=BIG + pool - 16) == INVALID
    assert append(desc(kv_fp8=True), ks=P, vs=P, kp=BIG, vp=BIG + pool) == INVALID
    s = dict(ks=P, vs=P, v=3 * BIG)
    assert read(d, k=P + pool - 16, **s) == INVALID


def test_decode_refuses():
    s = dict(ks=P, vs=P)
    for change in (dict(ws_bytes=100), dict(kp=P + 8), dict(q=None), dict(out=P + 8), dict(si=P),
                   dict(so=P, stride=999)):
        assert decode(desc(**FP4), **s, **change) == INVALID


def test_workspace_follows_the_form():
    big = dict(num_seqs=64, max_seq_len=8192, max_pages_per_seq=512, num_pages=40000)
    for scores in (False, True):
        assert q.paged_decode_workspace_size(desc(**FP4, **big), scores) > 0


def test_binding_refuses():
    d = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64, kv_fp4=True)
    with pytest.raises(ValueError, match="one form"):
        q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64, kv_fp8=True, kv_fp4=True)
    pool = torch.zeros(q.paged_pool_shape(d), dtype=torch.uint8)
    rows = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    table, s = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, 2)
    with pytest.raises(ValueError, match="k_out and v_out"):
        q.paged_kv_read(d, pool, pool, i32, table, None, None, k_scale=s, v_scale=s)
    with pytest.raises((ValueError, TypeError)):   # tensors of the host
        q.paged_kv_read(d, pool, pool, i32, table, rows, rows.clone(), k_scale=s, v_scale=s)
    with pytest.raises(TypeError, match="k_out"):
        q.paged_kv_read(d, pool, pool, i32, table, [1], rows, k_scale=s, v_scale=s)
    with pytest.raises((ValueError, TypeError)):
        q.paged_kv_append(d, rows, rows, i32, table, pool, pool.clone(), k_scale=s, v_scale=s)


@pytest.mark.gpu
def test_binding_refuses_wrong_pools():
    d = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64, kv_fp4=True)
    z = lambda *shape, **k: torch.zeros(*shape, device="cuda", **k)
    pool = z(q.paged_pool_shape(d), dtype=torch.uint8)
    rows, i32 = z(2, 2, 64, dtype=torch.bfloat16), z(2, dtype=torch.int32)
    table, s = z(2, 2, dtype=torch.int32), torch.ones(2, 2, device="cuda")
    for bad in (pool.view(8, 16, 2, 36), pool[:, :, :-1], pool.to(torch.int8), pool[:7], pool.transpose(0, 1),
                pool.cpu(), None):
        with pytest.raises((ValueError, TypeError)):
            q.paged_kv_read(d, bad, pool, i32, table, rows, rows.clone(), k_scale=s, v_scale=s)
    for kw in (dict(), dict(k_scale=s), dict(k_scale=s, v_scale=s[:1])):
        with pytest.raises(ValueError):
            q.paged_kv_read(d, pool, pool, i32, table, rows, rows.clone(), **kw)
    with pytest.raises(ValueError, match="start_pos"):
        q.paged_kv_read(d, pool, pool, i32[:1], table, rows, rows.clone(), k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="v_out"):
        q.paged_kv_read(d, pool, pool, i32, table, rows, z(3, 2, 64, dtype=torch.bfloat16), k_scale=s,
                        v_scale=s)
