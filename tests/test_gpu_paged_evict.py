"""GPU parity of quail_paged_kv_evict (eviction by accumulated attention weight) against the
oracle, bit for bit; and the paged operators run one after the other, as they are used."""
import math

import numpy as np
import pytest
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged
from paged_util import DEV, Cache, block_table, check_decode, f64, run_decode

pytestmark = pytest.mark.gpu

CASES = {
    "ragged": ([0, 1, 5, 40, 41, 100, 333, 1000, 2049], 40, 8),
    "all_recent": ([10, 90, 300], 50, 50),
    "no_recent": ([10, 90, 300], 50, 0),
    "one_place": ([1, 2, 700], 1, 0),
    "one_recent": ([1, 2, 700], 1, 1),
    "under_budget": ([5, 60, 64], 64, 3),
    "empty": ([0, 0], 16, 4),
    "larger": ([512, 511, 513, 2048, 2000], 512, 100),
    "past_one_launch": ([600, 2048], 513, 100),
}


def ok():
    torch.cuda.synchronize()
    st = q.get_device_error()
    assert st == q.QUAIL_OK, q.status_string(st)


def scores_for(lens, hkv, width, kind, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(len(lens), hkv, width, generator=gen)
    if kind == "heavy":                      # many exact zeros, a few large
        return torch.where(x < 0.5, torch.zeros_like(x), torch.exp(3 * x))
    if kind == "ties":
        return (x * 2).round()
    if kind == "equal":
        return torch.ones_like(x)
    if kind == "special":                    # NaN, infinities, signed zeros, subnormals
        pick = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-42, -1e-42, 1.0])
        return pick[torch.randint(0, 8, x.shape, generator=gen)]
    return x


def run(cache, score, budget, recent, dst=None, score_stride=None, dst_table=None, max_len=None):
    """dst None: another pool; "same": fresh pages of the cache's own pool."""
    B, hkv, d = len(cache.lens), cache.k.shape[2], cache.k.shape[3]
    page, dt = cache.page, cache.k.dtype
    fresh = [min(n, budget) for n in cache.lens]
    table, pages = block_table(fresh, page, np.random.default_rng(1),
                               width=-(-budget // page))
    if dst == "same":
        table = np.where(table >= 0, table + cache.pages, table).astype(np.int32)
        total = cache.pages + pages
        grown = [torch.zeros(total, page, hkv, d, dtype=torch.bfloat16, device=DEV).to(dt)
                 for _ in range(2)]
        for g, x in zip(grown, (cache.k, cache.v)):
            g.view(torch.uint8)[:cache.pages] = x.view(torch.uint8)
        cache.k, cache.v = grown
        cache.pages = total
        k_dst, v_dst = grown
    else:
        k_dst = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device=DEV).to(dt)
        v_dst = k_dst.clone()
    if dst_table is not None:
        table = dst_table(table)
    desc = cache.desc(2 * hkv, max_len)
    kept = torch.full((B, hkv, budget), -9, dtype=torch.int32, device=DEV)
    new = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    out = torch.full((B, hkv, score_stride or budget), -9.0, device=DEV)
    ws = torch.full((q.paged_evict_workspace_size(desc, k_dst.shape[0]),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    q.paged_kv_evict(desc, budget, recent, cache.k, cache.v, cache.table, cache.seq_lens,
                     score.to(DEV), torch.from_numpy(table).to(DEV), k_dst, v_dst, kept, new, ws,
                     score_out=out)
    return kept, new, out, k_dst, v_dst, table


def raw(x):
    return x.view(torch.uint8).cpu().numpy().reshape(-1, x.shape[2], x.shape[3] * x.element_size())


def check(cache, score, budget, recent, got, only=None):
    kept, new, out, k_dst, v_dst, table = got
    kept, new, out = kept.cpu().numpy(), new.cpu().numpy(), out.cpu().numpy()
    src = [raw(x) for x in (cache.k, cache.v)]
    dst = [raw(x) for x in (k_dst, v_dst)]
    s = score.numpy()
    for b, n in enumerate(cache.lens):
        if only is not None and b not in only:
            continue
        m = min(n, budget)
        assert new[b] == m
        for g in range(s.shape[1]):
            want = paged.evict(s[b, g], n, budget, recent)
            np.testing.assert_array_equal(kept[b, g, :m], want)
            assert (kept[b, g, m:] == -1).all()
            np.testing.assert_array_equal(out[b, g, :m].view(np.int32), s[b, g, want].view(np.int32))
            assert (out[b, g, m:] == 0).all()
            a = paged.slots(cache.table_np[b], want, cache.page)
            z = paged.slots(table[b], np.arange(m), cache.page)
            for x, y in zip(src, dst):
                np.testing.assert_array_equal(y[z, g], x[a, g])


@pytest.mark.parametrize("most", [0, 3000, 20000])    # (0: the longest; see below)
@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "special"])
@pytest.mark.parametrize("fp8", [False, True])
def test_cases(name, kind, fp8, most):
    lens, budget, recent = CASES[name]
    most = most or max(lens)
    cache = Cache(lens, 2, 64 if fp8 else 128, 16, fp8, seed=3, width=max(1, -(-most // 16)))
    score = scores_for(lens, 2, max(most, 1) + 2, kind)
    got = run(cache, score, budget, recent, score_stride=budget + 7, max_len=most)
    ok()
    check(cache, score, budget, recent, got)


@pytest.mark.parametrize("lens,budget,recent,hkv", [
    ([70000], 3000, 64, 1),        # a cluster's CTAs share the keys
    ([170001, 20000], 9000, 100, 1),  # and do not hold all of them
    ([400003, 3, 262144], 30000, 1000, 1),
    ([5000] * 40, 1000, 16, 4),    # one CTA each
    ([20481, 20480, 4097], 20480, 0, 2),
    ([16384, 9000, 5], 1024, 100, 1),  # one launch of clusters of eight
    ([16000, 900, 1024], 1000, 990, 1),
    ([4096, 2049, 256, 300], 256, 17, 2),  # and of two
])
@pytest.mark.parametrize("kind", ["heavy", "normal", "equal"])
def test_long(lens, budget, recent, hkv, kind):
    cache = Cache(lens, hkv, 64, 256, True, seed=4)
    score = scores_for(lens, hkv, max(lens), kind, seed=len(lens))
    got = run(cache, score, budget, recent)
    ok()
    check(cache, score, budget, recent, got)


# max_seq_len 200: one launch; 3,000: one of clusters; 20,000: select and copy are two
@pytest.mark.parametrize("most", [200, 3000, 20000])
def test_same_pool_and_shared_source_pages(most):
    cache = Cache([200, 200, 90], 2, 128, 16, False, width=-(-most // 16))
    cache.table_np[1, :6] = cache.table_np[0, :6]       # a shared prefix
    cache.table.copy_(torch.from_numpy(cache.table_np))
    score = scores_for(cache.lens, 2, most, "normal")
    got = run(cache, score, 64, 8, dst="same", max_len=most)
    ok()
    check(cache, score, 64, 8, got)


@pytest.mark.parametrize("most", [200, 3000, 20000])
@pytest.mark.parametrize("where", ["twice", "itself", "held", "outside"])
def test_destination_pages_that_break_the_rules(where, most):
    """The sequences concerned end with -1 and nothing written there; the others are right."""
    cache = Cache([200, 150, 90], 2, 128, 16, False, width=-(-most // 16))
    score = scores_for(cache.lens, 2, most, "normal")
    held = int(cache.table_np[2, 1])

    def spoil(table):
        table = table.copy()
        if where == "twice":
            table[0, 2] = table[1, 3]
        elif where == "itself":
            table[1, 0] = table[1, 2]
        elif where == "held":
            table[1, 3] = held
        else:
            table[1, 0] = cache.pages
        return table

    before = cache.k.clone()
    got = run(cache, score, 64, 8, dst="same", dst_table=spoil, max_len=most)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    assert q.get_device_error() == q.QUAIL_OK
    hit = {0, 1} if where == "twice" else {1}
    for b in range(3):
        assert (int(got[1][b]) == -1) == (b in hit)
    check(cache, score, 64, 8, got, only=set(range(3)) - hit)
    assert torch.equal(cache.k[:before.shape[0]].view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("most", [100, 20000])
def test_many_sequences(most):
    """More tables than the blocks that look them over take at once; two sequences that claim
    one page."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 101, 700).tolist()
    lens[3], lens[699] = 80, 90
    cache = Cache(lens, 1, 64, 16, False, width=-(-most // 16))
    score = scores_for(lens, 1, most, "normal")

    def spoil(table):
        table = table.copy()
        table[699, 1] = table[3, 2]
        return table

    got = run(cache, score, 40, 4, dst="same", dst_table=spoil, max_len=most)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    new = got[1].tolist()
    assert new[3] == new[699] == -1
    check(cache, score, 40, 4, got, only=set(range(700)) - {3, 699})


@pytest.mark.parametrize("most", [200, 3000, 20000])
def test_bad_sources_and_lengths(most):
    cache = Cache([200, 150, 90, 60], 2, 128, 16, False, width=-(-most // 16))
    score = scores_for(cache.lens, 2, most, "normal")
    table = cache.table_np.copy()
    table[1, :] = -1
    cache.table = torch.from_numpy(table).to(DEV)
    cache.seq_lens = torch.tensor([200, 150, most + 1, -4], dtype=torch.int32,
                                  device=DEV)
    got = run(cache, score, 64, 8, max_len=most)
    torch.cuda.synchronize()
    assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
    assert got[1].tolist() == [64, -1, -1, -1]
    assert (got[0][2:] == -1).all()
    check(cache, score, 64, 8, got, only=[0])


def test_captured_graph_on_another_stream():
    cache = Cache([200, 150], 2, 128, 16, False)
    desc = cache.desc(4)
    score = scores_for(cache.lens, 2, 200, "normal").to(DEV)
    table, pages = block_table([64, 64], 16, np.random.default_rng(1))
    dst = torch.from_numpy(table).to(DEV)
    k, v = (torch.zeros(pages, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kept = torch.empty(2, 2, 64, dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(q.paged_evict_workspace_size(desc, pages), dtype=torch.uint8, device=DEV)
    call = lambda s=None: q.paged_kv_evict(desc, 64, 8, cache.k, cache.v, cache.table,  # noqa: E731
                                           cache.seq_lens, score, dst, k, v, kept, new, ws, stream=s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (5, 6):
        fresh = scores_for(cache.lens, 2, 200, "heavy", seed=seed)
        score.copy_(fresh)
        cache.lens = [200 - seed, 40]
        cache.seq_lens.copy_(torch.tensor(cache.lens, dtype=torch.int32))
        graph.replay()
        ok()
        out = torch.zeros(2, 2, 64)
        for b, n in enumerate(cache.lens):
            for g in range(2):
                want = paged.evict(fresh[b, g].numpy(), n, 64, 8)
                out[b, g, :len(want)] = fresh[b, g][torch.from_numpy(want)]
        check(cache, fresh, 64, 8, (kept, new, out, k, v, table))


def test_nothing_to_do():
    """No sequences at all, and sequences without tokens."""
    i32 = dict(dtype=torch.int32, device=DEV)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    pages = torch.zeros(3, 16, 2, 64, **bf)
    desc = q.make_paged_desc(0, 40, 3, 16, 3, 4, 2, 64)
    none = torch.zeros(0, **i32)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    q.paged_kv_append(desc, torch.zeros(0, 2, 64, **bf), torch.zeros(0, 2, 64, **bf), none,
                      torch.zeros(0, 3, **i32), pages, pages.clone())
    q.paged_decode_attn(desc, torch.zeros(0, 4, 64, **bf), pages, pages, torch.zeros(0, 3, **i32), none,
                        torch.zeros(0, 4, 64, **bf), ws, lse=torch.zeros(0, 4, device=DEV),
                        score_out=torch.zeros(0, 2, 40, device=DEV))
    q.attn_scores(torch.zeros(0, 4, 64, **bf), torch.zeros(0, 2, 64, **bf), torch.zeros(0, 4, device=DEV),
                  torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(0, 2, 40, device=DEV), 0, 0)
    q.paged_kv_evict(desc, 8, 2, pages, pages, torch.zeros(0, 3, **i32), none,
                     torch.zeros(0, 2, 40, device=DEV), torch.zeros(0, 1, **i32), pages.clone(),
                     pages.clone(), torch.zeros(0, 2, 8, **i32), torch.zeros(0, **i32), ws)
    # prompts of no new tokens, and positions that nothing is written to
    desc = q.make_paged_desc(2, 40, 3, 16, 3, 4, 2, 64)
    q.paged_kv_append(desc, torch.zeros(0, 2, 64, **bf), torch.zeros(0, 2, 64, **bf),
                      torch.zeros(2, **i32), torch.zeros(2, 3, **i32), pages, pages.clone(),
                      new_offsets=torch.zeros(3, **i32))
    ok()
    assert (pages == 0).all()


FIRST_CALL_IN_A_CAPTURE = """
import torch, prefill_only_cascade_gb300 as q
dev = "cuda"
bf, i32 = torch.bfloat16, torch.int32
k, v = (torch.randn(8, 16, 2, 128, device=dev).to(bf) for _ in range(2))
table = torch.arange(8, dtype=i32, device=dev)[None]
n = torch.tensor([100], dtype=i32, device=dev)
x = torch.randn(1, 8, 128, device=dev).to(bf)
desc = q.make_paged_desc(1, 128, 8, 16, 8, 8, 2, 128)
out, lse = torch.zeros(1, 8, 128, dtype=bf, device=dev), torch.zeros(1, 8, device=dev)
score = torch.zeros(1, 2, 128, device=dev)
ws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=dev)
flat, off = k.view(128, 2, 128), torch.tensor([0, 100], dtype=i32, device=dev)
q_all, l_all = torch.randn(100, 8, 128, device=dev).to(bf), torch.full((100, 8), 6.0, device=dev)
votes = torch.zeros(1, 2, 128, device=dev)
kd, vd = torch.zeros(2, 16, 2, 128, dtype=bf, device=dev), torch.zeros(2, 16, 2, 128, dtype=bf, device=dev)
kept, new = torch.zeros(1, 2, 20, dtype=i32, device=dev), torch.zeros(1, dtype=i32, device=dev)
to = torch.arange(2, dtype=i32, device=dev)[None]
ews = torch.empty(q.paged_evict_workspace_size(desc, 2), dtype=torch.uint8, device=dev)
torch.cuda.synchronize()
def step():
    q.paged_kv_append(desc, x[:, :2], x[:, 2:4], n - 1, table, k, v)
    q.paged_decode_attn(desc, x, k, v, table, n, out, ws, lse=lse, score_out=score)
    q.attn_scores(q_all, flat[:100], l_all, off, off, votes, 100, 100, window=16)
    q.paged_kv_evict(desc, 20, 4, k, v, table, n, votes, to, kd, vd, kept, new, ews)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
assert q.get_device_error() == 0
got = [t.clone() for t in (out, lse, score, votes, kept, new, kd, vd)]
step()
torch.cuda.synchronize()
assert q.get_device_error() == 0
assert all(torch.equal(a, b) for a, b in zip(got, (out, lse, score, votes, kept, new, kd, vd)))
assert new.item() == 20 and float(out.abs().sum()) > 0
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, timeout=240,
                         capture_output=True, text=True)
    assert run.returncode == 0 and "same" in run.stdout, run.stdout + run.stderr


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_evict_then_tokens(fp8):
    """Prefill; prompts into pages; the weight their tokens receive; eviction; then tokens one
    by one, appended, attended to and weighed - against the same steps of the oracle."""
    hq, hkv, d, page, budget, recent = 8, 2, 128, 16, 96, 16
    lens = [150, 40, 260, 97]
    B, T, steps = len(lens), sum(lens), 5
    gen = torch.Generator().manual_seed(11)
    x = lambda *s: torch.randn(*s, generator=gen).bfloat16()  # noqa: E731
    qs, ks, vs = x(T, hq, d), x(T, hkv, d), x(T, hkv, d)
    off_np = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    off = torch.from_numpy(off_np).to(DEV)
    gq, gk, gv = qs.to(DEV), ks.to(DEV), vs.to(DEV)
    out, lse = torch.empty_like(gq), torch.empty(T, hq, device=DEV)
    k_amax, v_amax = (torch.empty(B, hkv, device=DEV) for _ in range(2))
    ws = torch.empty(q.causal_prefill_workspace_size(B, T, max(lens), hq, hkv, d),
                     dtype=torch.uint8, device=DEV)
    q.causal_prefill_attn(gq, gk, gv, off, out, max(lens), lse=lse, workspace=ws, k_amax=k_amax,
                          v_amax=v_amax)
    # one pool: pages of the prompts, and pages for what is kept with room for the new tokens
    first, n1 = block_table(lens, page, np.random.default_rng(0))
    second, n2 = block_table([min(n, budget) + steps for n in lens], page, np.random.default_rng(1))
    second = np.where(second >= 0, second + n1, second).astype(np.int32)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kp, vp = (torch.zeros(n1 + n2, page, hkv, d, dtype=torch.bfloat16, device=DEV).to(dt)
              for _ in range(2))
    # room above the prompt's largest value for later tokens
    scales = dict(k_scale=k_amax * (2 / 448), v_scale=v_amax * (2 / 448)) if fp8 else {}
    t1, t2 = torch.from_numpy(first).to(DEV), torch.from_numpy(second).to(DEV)
    desc = q.make_paged_desc(B, max(lens), n1 + n2, page, first.shape[1], hq, hkv, d, kv_fp8=fp8)
    q.paged_kv_append(desc, gk, gv, torch.zeros(B, dtype=torch.int32, device=DEV), t1, kp, vp,
                      new_offsets=off, **scales)
    score = torch.zeros(B, hkv, max(lens), device=DEV)
    q.attn_scores(gq, gk, lse, off, off, score, max(lens), max(lens), window=32)
    kept = torch.empty(B, hkv, budget, dtype=torch.int32, device=DEV)
    n = torch.empty(B, dtype=torch.int32, device=DEV)
    cap = budget + steps
    weight = torch.empty(B, hkv, cap, device=DEV)
    ews = torch.empty(q.paged_evict_workspace_size(desc, n1 + n2), dtype=torch.uint8, device=DEV)
    q.paged_kv_evict(desc, budget, recent, kp, vp, t1, torch.tensor(lens, dtype=torch.int32, device=DEV),
                     score, t2, kp, vp, kept, n, ews, score_out=weight)
    ok()
    # the oracle's choice, where no score lies within rounding of the threshold
    s64, l64 = f64(score), f64(lse)
    for b, L in enumerate(lens):
        r = slice(off_np[b], off_np[b + 1])
        ref = paged.scores(f64(qs)[r], f64(ks)[r], l64[r], 1 / math.sqrt(d), True, 32)
        assert np.allclose(s64[b][:, :L], ref, rtol=1e-4)
        for g in range(hkv):
            want = paged.evict(s64[b, g], L, budget, recent)
            np.testing.assert_array_equal(kept[b, g].cpu().numpy()[:len(want)], want)
    assert n.tolist() == [min(L, budget) for L in lens]

    cut = Cache([min(L, budget) for L in lens], hkv, d, page, fp8)
    desc = q.make_paged_desc(B, cap, n1 + n2, page, second.shape[1], hq, hkv, d, kv_fp8=fp8)
    for step in range(steps):
        nk, nv, nq = x(B, hkv, d).to(DEV), x(B, hkv, d).to(DEV), x(B, hq, d).to(DEV)
        q.paged_kv_append(desc, nk, nv, n, t2, kp, vp, **scales)
        n += 1
        before = weight.clone()
        dws = torch.empty(q.paged_decode_workspace_size(desc, True), dtype=torch.uint8, device=DEV)
        o, l_ = torch.empty(B, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, hq, device=DEV)
        q.paged_decode_attn(desc, nq, kp, vp, t2, n, o, dws, lse=l_, score_in=weight,
                            score_out=weight, **scales)
        ok()
        cut.lens = n.tolist()
        cut.table_np, cut.k64, cut.v64 = second, f64(kp).reshape(-1, hkv, d), f64(vp).reshape(-1, hkv, d)
        if fp8:
            cut.ks64, cut.vs64 = f64(scales["k_scale"]), f64(scales["v_scale"])
        check_decode(cut, nq, hq, o, l_)
        for b, L in enumerate(cut.lens):
            k, v = cut.rows(b)
            w = paged.decode(f64(nq)[b], k, v, 1 / math.sqrt(d))[2]
            assert np.allclose(f64(weight - before)[b][:, :L], w, rtol=1e-3, atol=1e-5)
            assert (weight[b, :, L:] == 0).all()
            # the newest row is the one appended
            at = paged.slots(second[b], [L - 1], page)[0]
            got = kp.view(torch.uint8).view(-1, hkv, d * kp.element_size())[at]
            if not fp8:
                assert torch.equal(got.view(torch.bfloat16), nk[b])
