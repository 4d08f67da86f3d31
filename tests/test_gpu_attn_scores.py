"""GPU parity of quail_attn_scores (the attention weight that keys receive from many queries)
against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged
from paged_util import DEV, U32, f64

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    st = q.get_device_error()
    assert st == q.QUAIL_OK, q.status_string(st)


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def make(nq, nk, hq, hkv, d, seed, causal, scale):
    """Queries, keys and the lse of softmax attention between them (fp32, rounded)."""
    gen = torch.Generator().manual_seed(seed)
    qs = (torch.randn(sum(nq), hq, d, generator=gen) * 1.5).bfloat16()
    ks = torch.randn(sum(nk), hkv, d, generator=gen).bfloat16()
    lse, q0, k0 = [], 0, 0
    for a, b in zip(nq, nk):
        z = torch.einsum("ihd,jhd->ihj", qs[q0:q0 + a].double(),
                         ks[k0:k0 + b].double().repeat_interleave(hq // hkv, 1)) * scale
        if causal:
            see = torch.ones(a, b, dtype=torch.bool).tril(b - a)
            z = z.masked_fill(~see[:, None], -math.inf)
        lse.append(torch.logsumexp(z, -1) if b else torch.full((a, hq), -math.inf))
        q0, k0 = q0 + a, k0 + b
    return qs, ks, torch.cat(lse).float() if lse else torch.zeros(0, hq)


def check(score, qs, ks, lse, nq, nk, scale, causal, window, base=None):
    """|error| per term: the score's (d + 6) u of its magnitudes in log2 units, the lse's
    rounding and its product with log2(e) (3 u), exp2's 2^-22; the sums are compensated per 128
    queries, within which 32 terms are added one after the other (32 u)."""
    got, qn, kn, ln = f64(score), f64(qs), f64(ks), f64(lse)
    hq, hkv, d = qn.shape[1], kn.shape[1], qn.shape[2]
    q0 = k0 = 0
    for s, (a, b) in enumerate(zip(nq, nk)):
        if b:
            k, l_ = kn[k0:k0 + b], ln[q0:q0 + a]
            ref = paged.scores(qn[q0:q0 + a], k, l_, scale, causal, window)
            top = 0.0
            if a:
                top = scale * math.log2(math.e) * max(
                    np.max(np.abs(qn[q0:q0 + a, h]) @ np.abs(k[:, h // (hq // hkv)]).T)
                    for h in range(hq))
            fin = np.abs(l_[np.isfinite(l_)])
            rel = math.log(2) * ((d + 6) * U32 * top + 3 * U32 * 1.45 * (fin.max() if fin.size else 0)) \
                + 2.0 ** -22 + 48 * U32
            start = 0.0 if base is None else f64(base)[s][:, :b]
            tol = rel * ref + 2 * U32 * np.abs(start + ref) + 1e-36
            err = np.abs(got[s][:, :b] - start - ref)
            assert (err <= tol).all(), (s, err.max(), (err / np.maximum(tol, 1e-300)).max())
        assert (got[s][:, b:] == -3.0).all()
        q0, k0 = q0 + a, k0 + b


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (4, 1), (16, 2), (16, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (True, 200), (False, 0), (False, 33)])
def test_heads_masks_windows(hq, hkv, d, causal, window):
    nk = [1, 2, 127, 128, 129, 0, 300, 33]
    nq = nk if causal else [4, 0, 130, 1, 17, 3, 260, 0]
    scale = 1 / math.sqrt(d)
    qs, ks, lse = make(nq, nk, hq, hkv, d, hq + d, causal, scale)
    score = torch.full((len(nk), hkv, max(nk) + 3), -3.0, device=DEV)
    base = torch.rand(len(nk), hkv, max(nk) + 3, device=DEV)
    base_or_none = base if window else None
    q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(nq), offsets(nk), score, max(nq),
                  max(nk), causal=causal, window=window, score_in=base_or_none)
    ok()
    check(score, qs, ks, lse, nq, nk, scale, causal, window, base_or_none)


@pytest.mark.parametrize("nq,nk", [([700], [1300]), ([1300], [700]), ([0, 0], [5, 600]), ([3], [0])])
def test_causal_with_other_lengths(nq, nk):
    """Bottom-right aligned: more keys than queries, and queries that see nothing."""
    scale = 0.1
    qs, ks, lse = make(nq, nk, 4, 2, 64, 5, True, scale)
    score = torch.full((len(nk), 2, max(nk) + 3), -3.0, device=DEV)
    q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(nq), offsets(nk), score, max(nq),
                  max(nk), softmax_scale=scale)
    ok()
    check(score, qs, ks, lse, nq, nk, scale, True, 0)


@pytest.mark.parametrize("window", [20, 40, 100])
def test_long_runs_of_key_tiles(window):
    """Many sequences: a CTA takes up to 16 key tiles of one, with one, two or four query tiles."""
    nk = [2100, 1] + [2049 + 3 * i for i in range(38)]
    scale = 1 / math.sqrt(64)
    gen = torch.Generator().manual_seed(12)
    qs = torch.randn(sum(nk), 16, 64, generator=gen).bfloat16()
    ks = torch.randn(sum(nk), 4, 64, generator=gen).bfloat16()
    lse = 7 + torch.rand(sum(nk), 16, generator=gen)     # as good as any
    score = torch.full((len(nk), 4, max(nk) + 3), -3.0, device=DEV)
    q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(nk), offsets(nk), score, max(nk),
                  max(nk), window=window)
    ok()
    check(score, qs, ks, lse, nk, nk, scale, True, window)


def test_few_keys_many_queries():
    """Query tiles split over a cluster; the same bits every time."""
    nq, nk, scale = [5000, 1], [100, 40], 1 / math.sqrt(128)
    qs, ks, lse = make(nq, nk, 8, 2, 128, 6, False, scale)
    args = [qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(nq), offsets(nk)]
    runs = []
    for _ in range(3):
        score = torch.full((2, 2, 103), -3.0, device=DEV)
        q.attn_scores(*args, score, 5000, 100, causal=False)
        ok()
        runs.append(score)
    check(runs[0], qs, ks, lse, nq, nk, scale, False, 0)
    assert all(torch.equal(r, runs[0]) for r in runs)


def test_strides_and_garbage_between():
    """q and k as columns of one fused projection; rows of NaN before, between and after."""
    n, hq, hkv, d = [60, 200], 8, 2, 128
    scale = 1 / math.sqrt(d)
    qs, ks, lse = make(n, n, hq, hkv, d, 7, True, scale)
    row = torch.full((300, (hq + 2 * hkv) * d), math.nan).bfloat16()
    all_lse = torch.full((300, hq), math.nan)
    at = torch.cat([torch.arange(10, 70), torch.arange(90, 290)])
    row[at, :hq * d], row[at, hq * d:(hq + hkv) * d] = qs.flatten(1), ks.flatten(1)
    all_lse[at] = lse
    row = row.to(DEV)
    score = torch.full((3, hkv, 203), -3.0, device=DEV)
    # three ranges that follow one another; the middle one is the gap, of NaN rows
    off = torch.tensor([10, 70, 90, 290], dtype=torch.int32, device=DEV)
    q.attn_scores(row[:, :hq * d].view(300, hq, d), row[:, hq * d:(hq + hkv) * d].view(300, hkv, d),
                  all_lse.to(DEV), off, off, score, 200, 200)
    ok()
    assert torch.isnan(score[1, :, :20]).all() and (score[1, :, 20:] == -3).all()
    check(score[[0, 2]], qs, ks, lse, n, n, scale, True, 0)


def test_after_prefill():
    """With the lse that the prefill writes: each query's weights sum to 1."""
    hq, hkv, d, S, L = 8, 2, 128, 3, 300
    x = lambda *s: torch.randn(*s, device=DEV).bfloat16()  # noqa: E731
    qs, ks, vs = x(S * L, hq, d), x(S * L, hkv, d), x(S * L, hkv, d)
    off = torch.arange(S + 1, dtype=torch.int32, device=DEV) * L
    out, lse = torch.empty_like(qs), torch.empty(S * L, hq, device=DEV)
    ws = torch.empty(q.causal_prefill_workspace_size(S, S * L, L, hq, hkv, d), dtype=torch.uint8,
                     device=DEV)
    q.causal_prefill_attn(qs, ks, vs, off, out, L, lse=lse, workspace=ws)
    score = torch.zeros(S, hkv, L, device=DEV)
    q.attn_scores(qs, ks, lse, off, off, score, L, L)
    ok()
    total = score.sum(-1)
    assert torch.allclose(total, torch.full_like(total, L * hq / hkv), rtol=1e-3)
    assert torch.allclose(score[:, :, L - 1].sum(), torch.exp(
        (qs[L - 1::L].float().view(S, hkv, hq // hkv, d) * ks[L - 1::L].float()[:, :, None]).sum(-1)
        / math.sqrt(d) - lse[L - 1::L].view(S, hkv, hq // hkv)).sum(), rtol=1e-4)


def test_after_cascade():
    """The weight that anchors receive from all tokens of their suffixes, whose lse (over the
    anchor and the suffix itself) the cascade wrote."""
    import workloads
    from parity_util import run_cascade

    lay = workloads.layout_from_lengths([300, 0, 77], [3, 1, 2], [90, 5, 40, 9, 120, 3])
    hq, hkv, d = 8, 2, 128
    cfg = workloads.AttnConfig("scores", 3, (0, 0), 0, (0, 0), hq, hkv, d, False, 3)
    t = workloads.make_attention_inputs(cfg, lay, DEV)
    _, lse = run_cascade((hq, hkv, d), lay, t)
    q_off = t["suffix_offsets"][t["anchor_suffix_ptr"].long()].contiguous()
    score = torch.full((3, hkv, 303), -3.0, device=DEV)
    q.attn_scores(t["q_suf"], t["k_anc"], lse, q_off, t["anchor_offsets"], score, 135, 300,
                  causal=False)
    ok()
    check(score, t["q_suf"], t["k_anc"], lse, np.diff(q_off.cpu().numpy()).tolist(), [300, 0, 77],
          1 / math.sqrt(d), False, 0)


def test_lse_of_minus_infinity_gives_no_weight():
    n, scale = [150], 1 / 8
    qs, ks, lse = make(n, n, 2, 1, 64, 8, True, scale)
    lse[20:40, 0] = -math.inf
    score = torch.full((1, 1, 153), -3.0, device=DEV)
    q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(n), offsets(n), score, 150, 150)
    ok()
    check(score, qs, ks, lse, n, n, scale, True, 0)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 60), (True, 130), (True, 250), (False, 0)])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_queries_without_weight_may_hold_anything(causal, window, what):
    """Rows whose lse is -inf (padding, say) are left out although they hold NaN or infinities."""
    n, scale = [1200, 300], 1 / 8
    qs, ks, lse = make(n, n, 2, 1, 64, 11, causal, scale)
    for rows in (slice(0, 3), slice(700, 900), slice(1100, 1101), slice(1190, 1210), slice(1499, 1500)):
        qs[rows, 1], lse[rows, 1] = what, -math.inf
    score = torch.full((2, 1, 1203), -3.0, device=DEV)
    q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), offsets(n), offsets(n), score, 1200, 1200,
                  causal=causal, window=window)
    ok()
    qs[lse == -math.inf] = 0    # for the bound's magnitudes
    check(score, qs, ks, lse, n, n, scale, causal, window)


def test_bad_offsets_are_left_out_and_reported():
    n, scale = [50, 60, 70], 1 / 8
    qs, ks, lse = make(n, n, 2, 1, 64, 9, True, scale)
    good = [0, 50, 110, 180]
    for bad in ([0, 50, 200, 180], [0, 50, 40, 180], [-5, 50, 110, 180]):
        score = torch.full((3, 1, 73), -3.0, device=DEV)
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        q.attn_scores(qs.to(DEV), ks.to(DEV), lse.to(DEV), off, off, score, 70, 70)
        torch.cuda.synchronize()
        assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
        for s in range(3):
            if bad[s:s + 2] != good[s:s + 2]:
                assert (score[s] == -3.0).all()
            else:
                ref = paged.scores(f64(qs)[bad[s]:bad[s + 1]], f64(ks)[bad[s]:bad[s + 1]],
                                   f64(lse)[bad[s]:bad[s + 1]], scale, True)
                assert np.allclose(f64(score)[s][:, :n[s]], ref, rtol=1e-4)


def test_captured_graph_on_another_stream():
    n, scale = [200, 90], 1 / 8
    qs, ks, lse = make(n, n, 4, 2, 64, 10, True, scale)
    args = [t.to(DEV) for t in (qs, ks, lse)] + [offsets(n), offsets(n)]
    score = torch.full((2, 2, 203), -3.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.attn_scores(*args, score, 200, 200, stream=side)
    side.synchronize()
    first = score.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.attn_scores(*args, score, 200, 200, score_in=score)
    score.copy_(first)
    graph.replay()
    ok()
    assert torch.equal(score[0, :, :200], 2 * first[0, :, :200])
    check(first, qs, ks, lse, n, n, scale, True, 0)
