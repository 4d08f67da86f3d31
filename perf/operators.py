"""Cases of the paged-cache operators: K/V rows written into pages, attention of one new token
over the pages, the attention weight that cached tokens receive, and eviction by that weight.

A case is a dict of plain values; `prepare` makes a user's tensors for it from a seed, `run`
makes one pass (the plain torch form, or with `own` the library's calls), `work` gives the
bytes and operations the pass cannot do without and `exact` the result in 64 bits.

Pages hold [page_size, Hkv, d] token rows; a block table names the pages of each sequence.
Lengths come from the case alone (its "lens" number), so that `work` knows them.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, lo=1, hi=1, lens=0, hq=32, hkv=8, d=128, page=64, fp8=False)
    c.update(kw)
    return c


def listed():
    return [
        # one new token per sequence of a decode batch, codes with the anchors' scales; k and v
        # are columns of one fused projection's rows
        _case("append_token_fp8", "append", seqs=96, lo=1, hi=1, past=2000, fused=True, fp8=True,
              page=16, lens=11),
        # the prefilled prompts of a batch moved into pages
        _case("append_prompts", "append", seqs=96, lo=128, hi=2048, past=0, fused=False, lens=12),
        # a single short conversation: latency
        _case("decode_one", "decode", seqs=1, lo=777, hi=777, scored=False, page=16, lens=21),
        # a ragged serving batch
        _case("decode_batch", "decode", seqs=64, lo=128, hi=4096, scored=False, lens=22),
        # one very long context, an odd length that ends inside a page
        _case("decode_long", "decode", seqs=1, lo=131007, hi=131007, scored=False, lens=23),
        # long anchors held as e4m3 codes, the weights of every step accumulated for eviction
        _case("decode_scored_fp8", "decode", seqs=32, lo=2048, hi=8192, scored=True, fp8=True,
              lens=24),
        # small heads without many sequences, weights accumulated
        _case("decode_scored_small", "decode", seqs=4, lo=64, hi=600, hq=4, hkv=1, d=64,
              scored=True, page=16, lens=25),
        # what the last 32 tokens of each prompt attend to: the usual vote before eviction
        _case("scores_window", "scores", seqs=64, lo=128, hi=2048, causal=True, window=32, lens=31),
        # the weight that every token of four prompts receives from all later ones
        _case("scores_full", "scores", seqs=4, lo=4096, hi=4096, causal=True, window=0, lens=32),
        # a join: the weight that anchor tokens receive from all tokens of their suffixes
        _case("scores_join", "scores", seqs=8, lo=1000, hi=1024, causal=False, window=0,
              qlo=2000, qhi=4000, lens=33),
        # a batch over its budget
        _case("evict_batch", "evict", seqs=32, lo=2500, hi=6000, budget=1024, recent=64, lens=41),
        # two very long caches of e4m3 codes
        _case("evict_long_fp8", "evict", seqs=2, lo=100000, hi=131000, budget=8192, recent=256,
              fp8=True, page=128, lens=42),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "scores", "evict", "evict"])
    hkv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 8, 16])
    c = dict(op=op, hkv=hkv, hq=hkv * group, d=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.4,
             lens=rng.randrange(1 << 30))
    if op == "append":
        c["hi"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4000)
        c["lo"] = rng.randint(0, c["hi"]) if c["hi"] > 1 else 1
        c["past"] = rng.choice([0, _log_int(rng, 1, 3000)])
        c["seqs"] = _log_int(rng, 1, max(1, min(256, 100_000 // (c["hi"] + c["past"]))))
        c["fused"] = rng.random() < 0.5
    elif op == "decode":
        c["hi"] = _log_int(rng, 1, 131_071)
        c["lo"] = rng.randint(max(1, c["hi"] // 16), c["hi"])
        c["seqs"] = _log_int(rng, 1, max(1, min(200, 200_000 // c["hi"])))
        c["scored"] = rng.random() < 0.5
    elif op == "scores":
        c["fp8"] = False
        c["causal"] = rng.random() < 0.7
        most = 256_000 // c["hq"]
        c["hi"] = _log_int(rng, 1, min(4000, most))
        c["lo"] = rng.randint(max(1, c["hi"] // 8), c["hi"])
        c["seqs"] = _log_int(rng, 1, max(1, min(64, most // c["hi"])))
        c["window"] = rng.choice([0, _log_int(rng, 1, 64)])
        if not c["causal"]:
            c["qhi"] = _log_int(rng, 1, min(2000, 3_000_000 // (c["seqs"] * c["hq"])))
            c["qlo"] = rng.randint(0, c["qhi"])
    else:
        c["hi"] = _log_int(rng, 8, 131_000)
        c["lo"] = rng.randint(max(1, c["hi"] // 8), c["hi"])
        c["budget"] = _log_int(rng, 1, min(8192, c["hi"]))
        c["seqs"] = _log_int(rng, 1, max(1, min(64, 200_000 // c["hi"], 90_000 // c["budget"])))
        c["recent"] = rng.randint(0, max(0, c["budget"] // 4))
    return c


def _lens(c):
    return np.random.default_rng(c["lens"]).integers(c["lo"], c["hi"] + 1, size=c["seqs"])


def _qlens(c):
    """Queries of each sequence in a `scores` case, before the window."""
    if c["causal"]:
        return _lens(c)
    return np.random.default_rng(c["lens"] + 1).integers(c["qlo"], c["qhi"] + 1, size=c["seqs"])


def _pairs(c):
    """(query token, key) pairs that a `scores` case sums."""
    nk, nq = _lens(c).astype(np.int64), _qlens(c).astype(np.int64)
    w = np.minimum(nq, c["window"]) if c["window"] else nq
    if not c["causal"]:
        return int((w * nk).sum()), int(w.sum())
    first = nk - w  # keys that every query of the window sees, less one
    return int((w * first + w * (w + 1) // 2).sum()), int(w.sum())


def work(c):
    n, hkv, hq, d = _lens(c).astype(np.int64), c["hkv"], c["hq"], c["d"]
    elt = 1 if c["fp8"] else 2
    rows = int(n.sum()) * hkv
    if c["op"] == "append":
        return {"bytes": 2 * rows * d * (2 + elt), "flops": 2 * rows * d if c["fp8"] else 0}
    if c["op"] == "decode":
        b = 2 * rows * d * elt + c["seqs"] * hq * (4 * d + 4) + (8 * rows if c["scored"] else 0)
        return {"bytes": b, "flops": 4 * d * int(n.sum()) * hq}
    if c["op"] == "scores":
        pairs, queries = _pairs(c)
        return {"bytes": 2 * rows * d + queries * hq * (2 * d + 4) + 8 * rows,
                "flops": 2 * d * pairs * hq}
    kept = int(np.minimum(n, c["budget"]).sum()) * hkv
    return {"bytes": 4 * rows + 4 * kept * d * elt
            + 8 * c["seqs"] * hkv * c["budget"], "flops": 0}


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape, scale=1.0):
    """N(0, scale^2) in bf16, drawn in slices."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        k = min(step, flat.numel() - i)
        flat[i:i + k] = torch.randn(k, generator=gen, device=DEV) * scale
    return out


def _codes(gen, *shape):
    """e4m3 codes of N(0, 1) values whose largest is near the format's largest."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        k = min(step, flat.numel() - i)
        x = torch.randn(k, generator=gen, device=DEV) * 90.0
        flat[i:i + k] = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return out


def _tables(gen, lens, page, spare=0):
    """Block table [B, P] int32 (a random order of the pool's pages; unused entries -1) and the
    number of pages in the pool."""
    need = (np.asarray(lens, np.int64) + page - 1) // page
    width, total = int(max(1, need.max())), int(need.sum()) + spare
    order = torch.randperm(max(total, 1), generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(width, device=DEV)[None] < torch.from_numpy(need).to(DEV)[:, None]
    table[used] = order[:int(need.sum())]
    return table, max(total, 1)


def _pool(gen, c, pages):
    shape = (pages, c["page"], c["hkv"], c["d"])
    return _codes(gen, *shape) if c["fp8"] else _randn(gen, *shape)


def _scales(gen, c):
    if not c["fp8"]:
        return None
    return (0.5 + torch.rand(c["seqs"], c["hkv"], generator=gen, device=DEV)) / 90.0


def _i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def _offsets(lens):
    return _i32(np.concatenate([[0], np.cumsum(lens)]))


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    n = _lens(c)
    hkv, hq, d, page = c["hkv"], c["hq"], c["d"], c["page"]
    s = {"case": c, "max_len": int(n.max())}
    if c["op"] == "append":
        t = int(n.sum())
        if c["fused"]:  # q, k and v side by side in one row
            row = _randn(gen, t, (hq + 2 * hkv) * d)
            s["k_new"] = row[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
            s["v_new"] = row[:, (hq + hkv) * d:].view(t, hkv, d)
        else:
            s["k_new"], s["v_new"] = _randn(gen, t, hkv, d), _randn(gen, t, hkv, d)
        s["new_offsets"] = None if c["lo"] == c["hi"] == 1 else _offsets(n)
        past = np.random.default_rng(int(seed)).integers(c["past"] // 2, c["past"] + 1, c["seqs"])
        s["start_pos"] = _i32(past)
        s["max_len"] = int(c["past"] + c["hi"])
        s["table"], pages = _tables(gen, np.full(c["seqs"], s["max_len"]), page)
        s["k_pages"] = torch.zeros(pages, page, hkv, d, device=DEV, dtype=torch.bfloat16)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        if c["fp8"]:
            s["k_pages"] = s["k_pages"].to(torch.float8_e4m3fn)
            s["v_pages"] = s["v_pages"].to(torch.float8_e4m3fn)
        s["k_scale"], s["v_scale"] = _scales(gen, c), _scales(gen, c)
    elif c["op"] == "decode":
        s["q"] = _randn(gen, c["seqs"], hq, d, scale=1.5)
        s["table"], pages = _tables(gen, n, page)
        s["k_pages"], s["v_pages"] = _pool(gen, c, pages), _pool(gen, c, pages)
        s["k_scale"], s["v_scale"] = _scales(gen, c), _scales(gen, c)
        s["seq_lens"] = _i32(n)
        s["out"] = torch.empty(c["seqs"], hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(c["seqs"], hq, device=DEV)
        if c["scored"]:
            s["score_in"] = torch.rand(c["seqs"], hkv, s["max_len"], generator=gen, device=DEV)
            s["score_out"] = torch.zeros_like(s["score_in"])
    elif c["op"] == "scores":
        nq = _qlens(c)
        s["q"] = _randn(gen, int(nq.sum()), hq, d, scale=1.5)
        s["k"] = _randn(gen, int(n.sum()), hkv, d)
        s["k_offsets"] = _offsets(n)
        s["q_offsets"] = s["k_offsets"] if c["causal"] else _offsets(nq)
        s["max_q"] = int(nq.max())
        s["lse"] = _lse(s, n, nq)  # an attention call's lse, natural log
        s["score_out"] = torch.zeros(c["seqs"], hkv, s["max_len"], device=DEV)
    else:
        s["table"], pages = _tables(gen, n, page)
        s["k_pages"], s["v_pages"] = _pool(gen, c, pages), _pool(gen, c, pages)
        s["seq_lens"] = _i32(n)
        # accumulated weights: a few heavy tokens, many light ones, some that received nothing
        x = torch.randn(c["seqs"], hkv, s["max_len"], generator=gen, device=DEV)
        s["score"] = torch.where(x < -1.5, torch.zeros_like(x), torch.exp(2.0 * x))
        kept = np.minimum(n, c["budget"])
        s["dst_table"], dst = _tables(gen, kept, page)
        s["k_dst"] = torch.zeros((dst,) + s["k_pages"].shape[1:], device=DEV,
                                 dtype=torch.bfloat16).to(s["k_pages"].dtype)
        s["v_dst"] = s["k_dst"].clone()
        s["kept"] = torch.empty(c["seqs"], hkv, c["budget"], dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.empty(c["seqs"], dtype=torch.int32, device=DEV)
        s["score_out"] = torch.empty(c["seqs"], hkv, c["budget"], device=DEV)
    return s


def _lse(s, n, nq):
    """lse [Tq, Hq] of softmax attention over the visible keys (16-bit products: an input)."""
    c = s["case"]
    group, out, q0, k0 = c["hq"] // c["hkv"], [], 0, 0
    for a, b in zip(nq, n):
        a, b = int(a), int(b)
        q = s["q"][q0:q0 + a].view(a, c["hkv"], group, c["d"]).permute(1, 2, 0, 3)
        k = s["k"][k0:k0 + b].permute(1, 0, 2)
        z = torch.matmul(q, k[:, None].transpose(-1, -2)).float() / math.sqrt(c["d"])
        if c["causal"]:
            z = z.masked_fill(torch.ones(a, b, dtype=torch.bool, device=DEV).triu(1 + b - a),
                              -math.inf)
        out.append(torch.logsumexp(z, -1).permute(2, 0, 1).reshape(a, c["hq"]))
        q0, k0 = q0 + a, k0 + b
    return torch.cat(out).contiguous()


# ------------------------------------------------------------------ the plain forms
def _slots(table, pos, page):
    """Row of the flattened pool [pages * page] for position `pos` [B, n] of each sequence."""
    return torch.gather(table.long(), 1, (pos // page).clamp(0, table.shape[1] - 1)) * page \
        + pos % page


def _plain_append(s):
    c = s["case"]
    t = s["k_new"].shape[0]
    row = torch.arange(t, device=DEV)
    if s["new_offsets"] is None:
        seq, pos = row, s["start_pos"].long()
    else:
        off = s["new_offsets"].long()
        seq = torch.searchsorted(off, row, right=True) - 1
        pos = s["start_pos"].long()[seq] + row - off[seq]
    slot = s["table"][seq, pos // c["page"]].long() * c["page"] + pos % c["page"]
    for name in ("k", "v"):
        x = s[name + "_new"]
        if c["fp8"]:
            x = x.float() / s[name + "_scale"][seq][:, :, None]
            x = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        flat = s[name + "_pages"].view(-1, c["hkv"], c["d"])
        if c["fp8"]:  # the same bytes: indexing of this type is not everywhere
            flat, x = flat.view(torch.uint8), x.view(torch.uint8)
        flat[slot] = x
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _rows(s, name, slot):
    """Gathered rows [B, n, Hkv, d] in 32 bits, dequantised."""
    flat = s[name + "_pages"].view(-1, s["case"]["hkv"], s["case"]["d"])
    if not s["case"]["fp8"]:
        return flat[slot].float()
    x = flat.view(torch.uint8)[slot].view(torch.float8_e4m3fn).float()
    return x * s[name + "_scale"][:, None, :, None]


def _plain_decode(s):
    c = s["case"]
    b, hkv, d = c["seqs"], c["hkv"], c["d"]
    group = c["hq"] // hkv
    pos = torch.arange(s["max_len"], device=DEV)[None].expand(b, -1)
    seen = pos < s["seq_lens"][:, None]
    slot = torch.where(seen, _slots(s["table"], pos, c["page"]), torch.zeros_like(pos))
    k = _rows(s, "k", slot).permute(0, 2, 3, 1)                   # [B, Hkv, d, n]
    q = s["q"].float().view(b, hkv, group, d)
    z = torch.matmul(q, k) / math.sqrt(d)
    del k
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    w = e / total
    v = _rows(s, "v", slot).masked_fill(~seen[:, :, None, None], 0.0).permute(0, 2, 1, 3)
    got = {"out": torch.matmul(w, v).reshape(b, c["hq"], d).bfloat16(),
           "lse": (m + torch.log(total)).reshape(b, c["hq"])}
    if c["scored"]:
        got["score"] = torch.where(seen[:, None], s["score_in"] + w.sum(2), s["score_out"])
    return got


def _padded(x, start, count, most):
    """Rows start[s] .. start[s] + count[s] of x as [S, most, ...] in 32 bits, and their mask."""
    i = torch.arange(most, device=DEV)[None]
    mask = i < count[:, None]
    row = torch.where(mask, start[:, None] + i, torch.zeros_like(i))
    return x[row].float(), mask


def _plain_scores(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    group = c["hq"] // hkv
    qo, ko = s["q_offsets"].long(), s["k_offsets"].long()
    nq, nk = qo[1:] - qo[:-1], ko[1:] - ko[:-1]
    w = nq.clamp(max=c["window"]) if c["window"] else nq
    most = min(c["window"], s["max_q"]) if c["window"] else s["max_q"]
    if most == 0:
        return {"score": s["score_out"]}
    q, qm = _padded(s["q"], qo[1:] - w, w, most)                  # [S, w, Hq, d]
    lse, _ = _padded(s["lse"], qo[1:] - w, w, most)
    k, km = _padded(s["k"], ko[:-1], nk, s["max_len"])
    q = q.view(c["seqs"], most, hkv, group, d).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.reshape(c["seqs"], hkv, group * most, d), k.permute(0, 2, 3, 1))
    z = z.view(c["seqs"], hkv, group, most, s["max_len"]).div_(math.sqrt(d))
    lse = lse.view(c["seqs"], most, hkv, group).permute(0, 2, 3, 1)
    see = qm[:, :, None] & km[:, None]
    if c["causal"]:  # query i of the window is token nk - w + i
        i = torch.arange(most, device=DEV)[None, :, None] + (nk - w)[:, None, None]
        see = see & (torch.arange(s["max_len"], device=DEV)[None, None] <= i)
    p = z.sub_(lse[..., None]).exp_().masked_fill_(~see[:, None, None], 0.0)
    total = p.sum((2, 3))
    return {"score": torch.where(km[:, None], total, s["score_out"])}


def _plain_evict(s):
    c = s["case"]
    b, hkv, budget = c["seqs"], c["hkv"], c["budget"]
    n = s["seq_lens"].long()[:, None, None]
    most = s["max_len"]
    pos = torch.arange(most, device=DEV)[None, None]
    new = n.clamp(max=budget)
    recent = new.clamp(max=c["recent"])
    rest = n - recent
    x = torch.nan_to_num(s["score"], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    x = x.masked_fill(pos >= rest, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    chosen = (pos < new - recent).expand_as(order)
    keep = torch.zeros(b, hkv, most, dtype=torch.bool, device=DEV).scatter_(-1, order, chosen)
    keep = keep | ((pos >= rest) & (pos < n))
    width = min(budget, most)
    kept = torch.sort(torch.where(keep, pos, most), dim=-1).values[..., :width]
    real = kept < most
    at = torch.where(real, kept, 0)
    score = torch.gather(s["score"], 2, at).masked_fill(~real, 0.0)
    flat = at.permute(0, 2, 1)                                     # [B, width, Hkv]
    src = _slots(s["table"], flat.reshape(b, -1), c["page"]).view(b, width, hkv)
    i = torch.arange(width, device=DEV)[None].expand(b, -1)
    dst = _slots(s["dst_table"], i, c["page"])
    ok = i < new[:, :, 0]
    head = torch.arange(hkv, device=DEV)
    for name in ("k", "v"):
        a, z = s[name + "_pages"], s[name + "_dst"]
        if c["fp8"]:
            a, z = a.view(torch.uint8), z.view(torch.uint8)
        rows = a.view(-1, hkv, c["d"])[src, head]
        z.view(-1, hkv, c["d"])[dst[ok]] = rows[ok]
    pad = (0, budget - width)
    return {"kept": torch.nn.functional.pad(torch.where(real, kept, -1), pad, value=-1).int(),
            "new_lens": new[:, 0, 0].int(), "k_dst": s["k_dst"], "v_dst": s["v_dst"],
            "score": torch.nn.functional.pad(score, pad)}


# ------------------------------------------------------------------ the library's calls
def _desc(q, s, table, pages, page):
    c = s["case"]
    return q.make_paged_desc(c["seqs"], s["max_len"], pages, page, table.shape[1], c["hq"],
                             c["hkv"], c["d"], kv_fp8=c["fp8"])


def _own_append(s):
    import prefill_only_cascade_gb300 as q
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"].shape[0], s["case"]["page"])
    q.paged_kv_append(s["desc"], s["k_new"], s["v_new"], s["start_pos"], s["table"], s["k_pages"],
                      s["v_pages"], new_offsets=s["new_offsets"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_decode(s):
    import prefill_only_cascade_gb300 as q
    scored = s["case"]["scored"]
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"].shape[0], s["case"]["page"])
        s["ws"] = torch.empty(q.paged_decode_workspace_size(s["desc"], with_scores=scored),
                              dtype=torch.uint8, device=DEV)
    q.paged_decode_attn(s["desc"], s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"],
                        s["out"], s["ws"], lse=s["lse"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"], score_in=s.get("score_in"),
                        score_out=s.get("score_out"))
    got = {"out": s["out"], "lse": s["lse"]}
    if scored:
        got["score"] = s["score_out"]
    return got


def _own_scores(s):
    import prefill_only_cascade_gb300 as q
    c = s["case"]
    q.attn_scores(s["q"], s["k"], s["lse"], s["q_offsets"], s["k_offsets"], s["score_out"],
                  s["max_q"], s["max_len"], causal=c["causal"], window=c["window"])
    return {"score": s["score_out"]}


def _own_evict(s):
    import prefill_only_cascade_gb300 as q
    c = s["case"]
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"].shape[0], c["page"])
        s["ws"] = torch.empty(q.paged_evict_workspace_size(s["desc"], s["k_dst"].shape[0]),
                              dtype=torch.uint8, device=DEV)
    q.paged_kv_evict(s["desc"], c["budget"], c["recent"], s["k_pages"], s["v_pages"], s["table"],
                     s["seq_lens"], s["score"], s["dst_table"], s["k_dst"], s["v_dst"], s["kept"],
                     s["new_lens"], s["ws"], score_out=s["score_out"])
    return {"kept": s["kept"], "new_lens": s["new_lens"], "k_dst": s["k_dst"],
            "v_dst": s["v_dst"], "score": s["score_out"]}


PLAIN = {"append": _plain_append, "decode": _plain_decode, "scores": _plain_scores,
         "evict": _plain_evict}
OWN = {"append": _own_append, "decode": _own_decode, "scores": _own_scores, "evict": _own_evict}


def run(s):
    if own:
        return OWN[s["case"]["op"]](s)
    return PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"append": _exact_append, "decode": _exact_decode, "scores": _exact_scores,
                "evict": _exact_evict}[c["op"]](s)


def _exact_append(s):
    c = s["case"]
    n, start = _lens(c), s["start_pos"].tolist()
    table, got, t = s["table"].tolist(), {}, 0
    where = []  # (sequence, slot) of each new row
    for b in range(c["seqs"]):
        for i in range(int(n[b])):
            p = start[b] + i
            where.append((b, table[b][p // c["page"]] * c["page"] + p % c["page"]))
            t += 1
    seq = torch.tensor([w[0] for w in where], device=DEV)
    slot = torch.tensor([w[1] for w in where], device=DEV)
    for name in ("k", "v"):
        x = s[name + "_new"].double()
        if c["fp8"]:
            x = (x / s[name + "_scale"].double()[seq][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        pages = s[name + "_pages"].double()
        pages.view(-1, c["hkv"], c["d"]).index_copy_(0, slot, x)
        got[name + "_pages"] = pages
    return got


def _exact_decode(s):
    c = s["case"]
    group, hkv, page = c["hq"] // c["hkv"], c["hkv"], c["page"]
    out = torch.zeros(c["seqs"], c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["seqs"], c["hq"], dtype=torch.float64, device=DEV)
    score = s["score_out"].double() if c["scored"] else None
    for b, n in enumerate(int(x) for x in _lens(c)):
        ids = s["table"][b, :(n + page - 1) // page].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_pages"][ids].double().reshape(-1, hkv, c["d"])[:n]
            kv.append(x * s[name + "_scale"][b].double()[None, :, None] if c["fp8"] else x)
        for g in range(hkv):
            h = slice(g * group, (g + 1) * group)
            z = s["q"][b, h].double() @ kv[0][:, g].T / math.sqrt(c["d"])
            lse[b, h] = torch.logsumexp(z, -1)
            w = torch.exp(z - lse[b, h, None])
            out[b, h] = w @ kv[1][:, g]
            if score is not None:
                score[b, g, :n] = s["score_in"][b, g, :n].double() + w.sum(0)
    return {"out": out, "lse": lse, **({"score": score} if score is not None else {})}


def _exact_scores(s):
    c = s["case"]
    if work(c)["flops"] > 1e12:
        return None  # many seconds of 64-bit products
    group = c["hq"] // c["hkv"]
    score = s["score_out"].double()
    q0 = k0 = 0
    for b, (a, n) in enumerate(zip(_qlens(c).tolist(), _lens(c).tolist())):
        w = min(a, c["window"]) if c["window"] else a
        q, l = s["q"][q0 + a - w:q0 + a].double(), s["lse"][q0 + a - w:q0 + a].double()
        k = s["k"][k0:k0 + n].double()
        see = torch.ones(w, n, dtype=torch.bool, device=DEV)
        if c["causal"]:
            see = see.tril(n - w)
        for g in range(c["hkv"]):
            total = torch.zeros(n, dtype=torch.float64, device=DEV)
            for h in range(g * group, (g + 1) * group):
                z = q[:, h] @ k[:, g].T / math.sqrt(c["d"])
                total += torch.where(see, torch.exp(z - l[:, h, None]), 0.0).sum(0)
            score[b, g, :n] = total
        q0, k0 = q0 + a, k0 + n
    return {"score": score}


def _exact_evict(s):
    c = s["case"]
    page, hkv, budget = c["page"], c["hkv"], c["budget"]
    k_dst, v_dst = s["k_dst"].double(), s["v_dst"].double()
    score = torch.zeros(c["seqs"], hkv, budget, dtype=torch.float64, device=DEV)
    host = s["score"].cpu().numpy()
    table, dst_table = s["table"].cpu().numpy(), s["dst_table"].cpu().numpy()
    for b, n in enumerate(int(x) for x in _lens(c)):
        new = min(n, budget)
        recent = min(c["recent"], new)
        i = np.arange(new)
        dst = torch.from_numpy(dst_table[b, i // page].astype(np.int64) * page + i % page).to(DEV)
        for g in range(hkv):
            x = host[b, g, :n - recent].astype(np.float64)
            best = np.argsort(-x, kind="stable")[:new - recent]
            kept = np.concatenate([np.sort(best), np.arange(n - recent, n)]).astype(np.int64)
            src = torch.from_numpy(table[b, kept // page].astype(np.int64) * page
                                   + kept % page).to(DEV)
            for pages, to in ((s["k_pages"], k_dst), (s["v_pages"], v_dst)):
                flat = pages.view(torch.uint8) if c["fp8"] else pages
                rows = flat.view(-1, hkv, c["d"])[src, g]
                rows = rows.view(pages.dtype).double()
                to.view(-1, hkv, c["d"])[dst, g] = rows
            score[b, g, :new] = torch.from_numpy(host[b, g, kept].astype(np.float64)).to(DEV)
    return {"kept": None, "new_lens": None, "k_dst": k_dst, "v_dst": v_dst, "score": score}
