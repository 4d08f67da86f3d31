"""Host-only checks of the paged cache's calls: the C ABI rejects bad arguments before any
launch, and the binding rejects tensors that the library would misread."""
import ctypes

import pytest
import torch

import prefill_only_cascade_gb300 as q

INVALID, UNSUPPORTED = q.QUAIL_ERR_INVALID_ARG, q.QUAIL_ERR_UNSUPPORTED
P = 0x10000                                    # a pointer that is never followed
BIG = 1 << 50


def desc(**over):
    a = dict(num_seqs=4, max_seq_len=1000, num_pages=100, page_size=16, max_pages_per_seq=63,
             num_q_heads=32, num_kv_heads=8, head_dim=128)
    a.update(over)
    return q.make_paged_desc(**a)


BAD_DESCS = [
    (dict(num_seqs=-1), INVALID), (dict(max_seq_len=-1), INVALID), (dict(num_pages=-1), INVALID),
    (dict(max_pages_per_seq=-1), INVALID), (dict(page_size=0), INVALID),
    (dict(page_size=-16), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED),
    (dict(num_q_heads=30), INVALID), (dict(num_kv_heads=0), INVALID),
    (dict(num_q_heads=256, num_kv_heads=8), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
    (dict(max_seq_len=1009), INVALID),          # more than the table's rows name
    (dict(max_seq_len=(1 << 30) + 1, max_pages_per_seq=1 << 27), UNSUPPORTED),
    (dict(num_seqs=1 << 24), UNSUPPORTED), (dict(num_seqs=1 << 21, max_pages_per_seq=1 << 11), UNSUPPORTED),
]


def append(d, **o):
    a = dict(num_new=4, k=P, v=P + (1 << 20), ks_=1024, vs_=1024, off=None, start=P, table=P, ks=None,
             vs=None, kp=P, vp=BIG)
    a.update(o)
    return q.lib.quail_paged_kv_append(
        None if d is None else ctypes.byref(d), a["num_new"], a["k"], a["v"], a["ks_"], a["vs_"],
        a["off"], a["start"], a["table"], a["ks"], a["vs"], a["kp"], a["vp"], None)


def decode(d, **o):
    a = dict(q=P, qs=4096, kp=P, vp=P, table=P, lens=P, ks=None, vs=None, out=P, lse=None, si=None,
             so=None, stride=0, ws=P, ws_bytes=BIG)
    a.update(o)
    return q.lib.quail_paged_decode_attn(
        None if d is None else ctypes.byref(d), a["q"], a["qs"], a["kp"], a["vp"], a["table"],
        a["lens"], a["ks"], a["vs"], a["out"], a["lse"], a["si"], a["so"], a["stride"], a["ws"],
        a["ws_bytes"], None)


def scores(**o):
    a = dict(seqs=2, tq=50, tk=60, mq=30, mk=40, hq=8, hkv=2, d=128, scale=0.0, causal=1, window=0,
             q=P, qs=1024, k=P, ks=256, lse=P, qo=P, ko=P, si=None, so=P, stride=40)
    a.update(o)
    return q.lib.quail_attn_scores(*a.values(), None)


def evict(d, **o):
    a = dict(budget=64, recent=8, kp=P, vp=BIG, table=P, lens=P, score=P, stride=1000, dst=P,
             dst_max=4, dst_pages=16, kd=2 * BIG, vd=3 * BIG, kept=P, new=P + 4096, so=None, so_stride=0,
             ws=P, ws_bytes=BIG)
    a.update(o)
    return q.lib.quail_paged_kv_evict(None if d is None else ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("change,expect", BAD_DESCS)
def test_bad_descriptors(change, expect):
    d = desc(**change)
    assert append(d, num_new=d.num_seqs) == expect
    assert decode(d) == expect
    assert evict(d) == expect
    assert q.paged_decode_workspace_size(d) == 0
    assert q.paged_evict_workspace_size(d, 4) == 0


def test_null_descriptor():
    assert append(None) == decode(None) == evict(None) == INVALID
    assert q.lib.quail_paged_decode_workspace_size(None, 0) == 0


@pytest.mark.parametrize("change", [
    dict(num_new=-1), dict(num_new=5), dict(ks_=1023), dict(ks_=1028), dict(vs_=1000), dict(k=None),
    dict(v=None), dict(start=None), dict(table=None), dict(kp=None), dict(vp=None), dict(k=P + 8),
    dict(vp=P + 4), dict(start=P + 2), dict(off=P + 1), dict(ks=P), dict(ks=P, vs=P),
    dict(vp=P), dict(vp=P + 1024),                 # K and V pages that overlap
])
def test_append_rejects(change):
    assert append(desc(), **change) == INVALID


def test_append_needs_scales_with_codes():
    for change in (dict(), dict(ks=P), dict(vs=P), dict(ks=P, vs=P + 2)):
        assert append(desc(kv_fp8=True), **change) == INVALID
    assert append(desc(num_seqs=0), num_new=3, off=P) == INVALID


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=P + 8), dict(qs=4095), dict(qs=4100), dict(kp=None), dict(vp=P + 8),
    dict(table=None), dict(lens=None), dict(lens=P + 2), dict(out=None), dict(out=P + 8),
    dict(lse=P + 2), dict(si=P), dict(so=P, stride=999), dict(so=P + 2, stride=1000), dict(ws=None),
    dict(ws=P + 8), dict(ws_bytes=100), dict(ks=P), dict(ks=P, vs=P),
])
def test_decode_rejects(change):
    assert decode(desc(), **change) == INVALID


def test_decode_workspace():
    d = desc()
    plain, scored = q.paged_decode_workspace_size(d), q.paged_decode_workspace_size(d, True)
    assert plain > 0 and scored >= plain + 4 * 32 * 1000 * 4
    assert decode(d, ws_bytes=plain - 1) == INVALID
    assert decode(d, so=P, stride=1000, ws_bytes=scored - 1) == INVALID
    assert decode(desc(kv_fp8=True)) == INVALID
    # it does not grow with the lengths without scores
    assert q.paged_decode_workspace_size(desc(max_seq_len=1 << 20, max_pages_per_seq=1 << 16)) < 8 << 20


@pytest.mark.parametrize("change,expect", [
    (dict(seqs=-1), INVALID), (dict(tq=-1), INVALID), (dict(tk=1 << 31), INVALID),
    (dict(mq=-1), INVALID), (dict(mk=-1), INVALID), (dict(window=-1), INVALID),
    (dict(causal=2), INVALID), (dict(seqs=0), INVALID), (dict(hq=7), INVALID),
    (dict(hkv=0), INVALID), (dict(hq=64, qs=8192), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(scale=-0.5), INVALID), (dict(scale=float("inf")), INVALID), (dict(qs=1023), INVALID),
    (dict(qs=1028), INVALID), (dict(ks=255), INVALID), (dict(stride=39), INVALID),
    (dict(q=None), INVALID), (dict(q=P + 8), INVALID), (dict(k=None), INVALID),
    (dict(lse=None), INVALID), (dict(lse=P + 2), INVALID), (dict(qo=None), INVALID),
    (dict(ko=P + 1), INVALID), (dict(so=None), INVALID), (dict(so=P + 2), INVALID),
    (dict(si=P + 2), INVALID), (dict(seqs=1 << 20, mk=1 << 20, stride=1 << 20), UNSUPPORTED),
    (dict(mk=(1 << 31) - 1000, stride=1 << 31), UNSUPPORTED),
])
def test_scores_rejects(change, expect):
    assert scores(**change) == expect


@pytest.mark.parametrize("change", [
    dict(budget=0), dict(recent=-1), dict(recent=65), dict(dst_max=3), dict(dst_max=-1),
    dict(dst_pages=-1), dict(stride=999), dict(so=P, so_stride=63), dict(kp=None), dict(vp=None),
    dict(table=None), dict(lens=None), dict(score=None), dict(dst=None), dict(kd=None), dict(vd=None),
    dict(kept=None), dict(new=None), dict(kp=P + 8), dict(kd=2 * BIG + 8), dict(score=P + 2),
    dict(kept=P + 2), dict(so=P + 2, so_stride=64), dict(ws=None), dict(ws=P + 4), dict(ws_bytes=100),
    dict(new=P), dict(new=P + 12),                          # overlaps seq_lens
    dict(so=P, so_stride=64), dict(so=P + 4000, so_stride=64),  # overlaps score
    dict(kd=P),                                             # one pool: V and the pages too
    dict(kd=P, vd=BIG),                                     # (16 pages there, 100 here)
    dict(kd=P + 4096), dict(vd=BIG + 4096), dict(vd=2 * BIG), dict(kd=BIG), dict(vd=P),
])
def test_evict_rejects(change):
    assert evict(desc(), **change) == INVALID


def test_evict_limits():
    assert evict(desc(), budget=1 << 30, dst_max=1 << 27, dst_pages=1 << 20, kd=1 << 60,
                 vd=1 << 61) != INVALID
    d = desc(num_seqs=1 << 10, num_kv_heads=32)
    assert evict(d, budget=(1 << 31) - 1, dst_max=1 << 10, kd=1 << 60, vd=1 << 61, new=1 << 59) == UNSUPPORTED
    assert evict(desc(num_seqs=1 << 12), dst_max=1 << 20, new=1 << 59) == UNSUPPORTED
    assert evict(desc(), budget=(1 << 30) + 1) == UNSUPPORTED


# ------------------------------------------------------------------ the binding
def cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_rejects_what_is_not_on_a_gpu():
    d = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64)
    bf, i32 = torch.bfloat16, torch.int32
    pages = cpu(8, 16, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        q.paged_kv_append(d, cpu(2, 2, 64, dtype=bf), cpu(2, 2, 64, dtype=bf), cpu(2, dtype=i32),
                          cpu(2, 2, dtype=i32), pages, pages)
    with pytest.raises(ValueError, match="workspace is required"):
        q.paged_decode_attn(d, cpu(2, 4, 64, dtype=bf), pages, pages, cpu(2, 2, dtype=i32),
                            cpu(2, dtype=i32), cpu(2, 4, 64, dtype=bf), None)
    with pytest.raises(ValueError, match="CUDA"):
        q.paged_decode_attn(d, cpu(2, 4, 64, dtype=bf), pages, pages, cpu(2, 2, dtype=i32),
                            cpu(2, dtype=i32), cpu(2, 4, 64, dtype=bf), cpu(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        q.attn_scores(cpu(5, 4, 64, dtype=bf), cpu(5, 2, 64, dtype=bf), cpu(5, 4), cpu(2, dtype=i32),
                      cpu(2, dtype=i32), cpu(1, 2, 5), 5, 5)
    with pytest.raises(ValueError, match="CUDA"):
        q.paged_kv_evict(d, 4, 1, pages, pages, cpu(2, 2, dtype=i32), cpu(2, dtype=i32), cpu(2, 2, 30),
                         cpu(2, 1, dtype=i32), pages, pages, cpu(2, 2, 4, dtype=i32), cpu(2, dtype=i32),
                         cpu(4096, dtype=torch.uint8))
