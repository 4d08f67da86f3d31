"""Cases of the paged cache held in 4 bits: rows quantised as they are appended and read back,
attention of one new token over the pages, reading ranges back to dense rows, and eviction.

A case is a dict of plain values; `prepare` makes a user's tensors for it from a seed, `run`
makes one pass (the plain torch form, or with `own` the library's calls), `work` gives the
bytes and operations the pass cannot do without and `exact` the result in 64 bits.

A row of d values (one token, one KV head) is held as d / 2 bytes of e2m1 codes (two a byte, the
even position in the low bits) and d / 16 e4m3 block scales; value = code * block scale * S with
one fp32 S for each sequence and KV head. A page is, for each KV head, the codes of page_size
tokens and then their block scales; a block table names the pages of each sequence.
Lengths come from the case alone (its "lens" number), so that `work` knows them. What is held in
pages is returned as the rows that it stands for.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 16           # values that share a block scale
E4M3_MAX = 448.0
E2M1_MAX = 6.0
WHOLE = E4M3_MAX * E2M1_MAX


# ------------------------------------------------------------------ the cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, lo=1, hi=1, lens=0, hq=32, hkv=8, d=128, page=64)
    c.update(kw)
    return c


def listed():
    return [
        # one new token per sequence of a decode batch, quantised into its page; k and v are
        # columns of one fused projection's rows
        _case("append_token", "append", seqs=96, lo=1, hi=1, past=2000, fused=True, page=16, lens=11),
        # the prefilled prompts of a batch moved into pages
        _case("append_prompts", "append", seqs=96, lo=128, hi=2048, past=0, fused=False, lens=12),
        # one prompt's rows read back for a second prefill behind it, not from its first token on
        _case("read_one", "read", seqs=1, lo=777, hi=777, past=100, page=16, lens=13),
        # the anchors of a join batch read back as dense rows for the cascade
        _case("read_anchors", "read", seqs=64, lo=4096, hi=4096, past=0, page=256, lens=14),
        # a single short conversation: latency
        _case("decode_one", "decode", seqs=1, lo=777, hi=777, scored=False, page=16, lens=21),
        # a ragged serving batch
        _case("decode_batch", "decode", seqs=64, lo=128, hi=4096, scored=False, lens=22),
        # many short sequences, sixteen query heads to a KV head
        _case("decode_short", "decode", seqs=181, lo=20, hi=83, hq=64, hkv=4, scored=False, page=16,
              lens=23),
        # one very long context, an odd length that ends inside a page
        _case("decode_long", "decode", seqs=1, lo=131007, hi=131007, scored=False, lens=24),
        # long anchors, the weights of every step accumulated for eviction
        _case("decode_scored", "decode", seqs=32, lo=2048, hi=8192, scored=True, page=128, lens=25),
        # small heads without many sequences, weights accumulated
        _case("decode_scored_small", "decode", seqs=4, lo=64, hi=600, hq=4, hkv=1, d=64,
              scored=True, page=16, lens=26),
        # a batch over its budget
        _case("evict_batch", "evict", seqs=32, lo=2500, hi=6000, budget=1024, recent=64, lens=41),
        # one conversation cut down between two turns
        _case("evict_one", "evict", seqs=1, lo=4000, hi=4000, budget=128, recent=32, page=16, lens=42),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "append", "read", "read", "decode", "decode", "decode", "evict"])
    hkv = rng.choice([1, 2, 3, 4, 8, 8])
    group = rng.choice([1, 2, 4, 4, 8, 16])
    c = dict(op=op, hkv=hkv, hq=hkv * group, d=rng.choice([64, 128, 128]),
             page=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(1 << 30))
    if op in ("append", "read"):
        c["hi"] = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4000)
        c["lo"] = rng.randint(0, c["hi"]) if c["hi"] > 1 else 1
        c["past"] = rng.choice([0, _log_int(rng, 1, 3000)])
        c["seqs"] = _log_int(rng, 1, max(1, min(256, 100_000 // (c["hi"] + c["past"]))))
        if op == "append":
            c["fused"] = rng.random() < 0.5
    elif op == "decode":
        c["hi"] = _log_int(rng, 1, 131_071)
        c["lo"] = rng.randint(max(1, c["hi"] // 16), c["hi"])
        c["seqs"] = _log_int(rng, 1, max(1, min(200, 200_000 // c["hi"])))
        c["scored"] = rng.random() < 0.5
    else:
        c["hi"] = _log_int(rng, 8, 131_000)
        c["lo"] = rng.randint(max(1, c["hi"] // 8), c["hi"])
        c["budget"] = _log_int(rng, 1, min(8192, c["hi"]))
        c["seqs"] = _log_int(rng, 1, max(1, min(64, 200_000 // c["hi"], 90_000 // c["budget"])))
        c["recent"] = rng.randint(0, max(0, c["budget"] // 4))
    return c


def _lens(c):
    n = np.random.default_rng(c["lens"]).integers(c["lo"], c["hi"] + 1, size=c["seqs"])
    n[0] = max(n[0], 1)
    return n


def work(c):
    n, hkv, hq, d = _lens(c).astype(np.int64), c["hkv"], c["hq"], c["d"]
    rows = int(n.sum()) * hkv
    held = d // 2 + d // BLOCK  # bytes of a row in a page
    if c["op"] == "append":     # the rows read, their pages written, and the rows read back
        return {"bytes": 2 * rows * (2 * d + held + 2 * d), "flops": 4 * rows * d}
    if c["op"] == "read":
        return {"bytes": 2 * rows * (held + 2 * d), "flops": 4 * rows * d}
    if c["op"] == "decode":
        return {"bytes": 2 * rows * held + c["seqs"] * hq * (4 * d + 4)
                + (8 * rows if c["scored"] else 0), "flops": 4 * d * int(n.sum()) * hq}
    kept = int(np.minimum(n, c["budget"]).sum()) * hkv  # moved, and read back from where they are
    return {"bytes": 4 * rows + 2 * kept * (2 * held + 2 * d) + 8 * c["seqs"] * hkv * c["budget"],
            "flops": 0}


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape, scale=1.0):
    """N(0, scale^2) in bf16, drawn in slices."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat, step = out.view(-1), 1 << 26
    for i in range(0, flat.numel(), step):
        k = min(step, flat.numel() - i)
        flat[i:i + k] = torch.randn(k, generator=gen, device=DEV) * scale
    return out


def _tables(gen, lens, page):
    """Block table [B, P] int32 (a random order of the pool's pages; unused entries -1) and the
    number of pages in the pool."""
    need = (np.asarray(lens, np.int64) + page - 1) // page
    width, total = int(max(1, need.max())), int(need.sum())
    order = torch.randperm(max(total, 1), generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(need), width), -1, dtype=torch.int32, device=DEV)
    used = torch.arange(width, device=DEV)[None] < torch.from_numpy(need).to(DEV)[:, None]
    table[used] = order[:int(need.sum())]
    return table, max(total, 1)


def _pool(gen, c, pages, filled=True):
    """A pool [pages, Hkv, bytes of a page's head]: codes and block scales of N(0, 1) rows, the
    largest of which are near what the two formats hold."""
    hkv, d, page = c["hkv"], c["d"], c["page"]
    pool = torch.zeros(pages, hkv, page * (d // 2 + d // BLOCK), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (hkv * page * d))
    for i in range(0, pages if filled else 0, step):
        k = min(step, pages - i)
        x = torch.randn(k, hkv, page, d, generator=gen, device=DEV)
        codes, blocks = _quantise(x, torch.full((1, 1, 1), 5.0 / WHOLE, device=DEV))
        pool[i:i + k, :, :page * d // 2] = codes.view(k, hkv, -1)
        pool[i:i + k, :, page * d // 2:] = blocks.view(k, hkv, -1)
    return pool


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
    # what 5 standard deviations need, more or less
    s["k_scale"] = (0.75 + 0.5 * torch.rand(c["seqs"], hkv, generator=gen, device=DEV)) * 5.0 / WHOLE
    s["v_scale"] = (0.75 + 0.5 * torch.rand(c["seqs"], hkv, generator=gen, device=DEV)) * 5.0 / WHOLE
    if c["op"] in ("append", "read"):
        t = int(n.sum())
        s["offsets"] = None if c["lo"] == c["hi"] == 1 else _offsets(n)
        past = np.random.default_rng(int(seed)).integers(c["past"] // 2, c["past"] + 1, c["seqs"])
        s["start_pos"] = _i32(past)
        s["max_len"] = int(c["past"] + c["hi"])
        s["table"], pages = _tables(gen, np.full(c["seqs"], s["max_len"]), page)
        s["k_pages"] = _pool(gen, c, pages, c["op"] == "read")
        s["v_pages"] = _pool(gen, c, pages, c["op"] == "read")
        s["k_out"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
        if c["op"] == "append" and c["fused"]:  # q, k and v side by side in one row
            row = _randn(gen, t, (hq + 2 * hkv) * d)
            s["k_new"] = row[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
            s["v_new"] = row[:, (hq + hkv) * d:].view(t, hkv, d)
        elif c["op"] == "append":
            s["k_new"], s["v_new"] = _randn(gen, t, hkv, d), _randn(gen, t, hkv, d)
        return s
    s["seq_lens"] = _i32(n)
    s["table"], pages = _tables(gen, n, page)
    s["k_pages"], s["v_pages"] = _pool(gen, c, pages), _pool(gen, c, pages)
    if c["op"] == "decode":
        s["q"] = _randn(gen, c["seqs"], hq, d, scale=1.5)
        s["out"] = torch.empty(c["seqs"], hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(c["seqs"], hq, device=DEV)
        if c["scored"]:
            s["score_in"] = torch.rand(c["seqs"], hkv, s["max_len"], generator=gen, device=DEV)
            s["score_out"] = torch.zeros_like(s["score_in"])
        return s
    # accumulated weights: a few heavy tokens, many light ones, some that received nothing
    x = torch.randn(c["seqs"], hkv, s["max_len"], generator=gen, device=DEV)
    s["score"] = torch.where(x < -1.5, torch.zeros_like(x), torch.exp(2.0 * x))
    new = np.minimum(n, c["budget"])
    s["dst_table"], dst = _tables(gen, new, page)
    s["k_dst"], s["v_dst"] = _pool(gen, c, dst, False), _pool(gen, c, dst, False)
    s["kept"] = torch.empty(c["seqs"], hkv, c["budget"], dtype=torch.int32, device=DEV)
    s["new_lens"] = torch.empty(c["seqs"], dtype=torch.int32, device=DEV)
    s["score_out"] = torch.empty(c["seqs"], hkv, c["budget"], device=DEV)
    s["offsets"], s["start_pos"] = _offsets(new), _i32(np.zeros(c["seqs"]))
    s["k_out"] = torch.empty(int(new.sum()), hkv, d, dtype=torch.bfloat16, device=DEV)
    s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ------------------------------------------------------------------ the plain forms
def _quantise(x, scale):
    """Rows x [..., d] in 32 bits under scale [...] -> packed codes [..., d / 2] and block scales
    [..., d / 16], as bytes. Quotients are rounded to 32 bits, then to the nearest code, ties to
    the even one; what is too large takes the largest."""
    x = x.unflatten(-1, (-1, BLOCK))
    t = x.abs().amax(-1) / (E2M1_MAX * scale)[..., None]
    blocks = t.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    b = blocks.float()
    y = (x / (b * scale[..., None])[..., None]).masked_fill((b == 0)[..., None], 0.0)
    a = y.abs().clamp(max=E2M1_MAX).nan_to_num(0.0)
    code = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, a.round() + 2, (a / 2).round() + 4))
    code = (code + 8 * (y < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), blocks.view(torch.uint8)


def _values(codes, blocks, scale):
    """The rows [..., d] that packed codes and block scales under scale [...] stand for, in 32 bits."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    grid = torch.cat([grid, -grid])
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    x = torch.index_select(grid, 0, code.flatten().int()).view(code.shape).unflatten(-1, (-1, BLOCK))
    b = blocks.view(torch.float8_e4m3fn).float() * scale[..., None]
    return (x * b[..., None]).flatten(-2)


def _parts(pool, c):
    """Codes [pages, Hkv, page, d / 2] and block scales [pages, Hkv, page, d / 16] of a pool."""
    cut, d = c["page"] * c["d"] // 2, c["d"]
    return (pool[:, :, :cut].unflatten(-1, (c["page"], d // 2)),
            pool[:, :, cut:].unflatten(-1, (c["page"], d // BLOCK)))


def _rows_of(s):
    """Sequence, page and place in it of every row of an append or a read."""
    row = torch.arange(s["k_out"].shape[0], device=DEV)
    if s["offsets"] is None:
        seq, pos = row, s["start_pos"].long()
    else:
        off = s["offsets"].long()
        seq = torch.searchsorted(off, row, right=True) - 1
        pos = s["start_pos"].long()[seq] + row - off[seq]
    page = s["case"]["page"]
    return seq, s["table" if s["case"]["op"] != "evict" else "dst_table"][seq, pos // page].long(), \
        pos % page


def _plain_put(x, pool, scale, where, c):
    seq, page, at = where
    codes, blocks = _quantise(x.float(), scale[seq])
    to_codes, to_blocks = _parts(pool, c)
    to_codes[page, :, at] = codes
    to_blocks[page, :, at] = blocks


def _plain_get(pool, scale, where, c):
    seq, page, at = where
    codes, blocks = _parts(pool, c)
    return _values(codes[page, :, at], blocks[page, :, at], scale[seq]).bfloat16()


def _plain_append(s):
    c, where = s["case"], _rows_of(s)
    _plain_put(s["k_new"], s["k_pages"], s["k_scale"], where, c)
    _plain_put(s["v_new"], s["v_pages"], s["v_scale"], where, c)
    return {"k": _plain_get(s["k_pages"], s["k_scale"], where, c),
            "v": _plain_get(s["v_pages"], s["v_scale"], where, c)}


def _plain_read(s):
    c, where = s["case"], _rows_of(s)
    return {"k": _plain_get(s["k_pages"], s["k_scale"], where, c),
            "v": _plain_get(s["v_pages"], s["v_scale"], where, c)}


def _dense(pool, scale, s, seen):
    """Rows [B, Hkv, n, d] of all sequences in 32 bits, zeros behind the last."""
    c = s["case"]
    pos = torch.arange(s["max_len"], device=DEV)[None].expand(c["seqs"], -1)
    page = torch.gather(s["table"].long(), 1, pos // c["page"]).clamp(min=0)
    codes, blocks = _parts(pool, c)
    at = pos % c["page"]
    x = _values(codes[page, :, at], blocks[page, :, at], scale[:, None].expand(-1, s["max_len"], -1))
    return x.masked_fill(~seen[:, :, None, None], 0.0).permute(0, 2, 1, 3)


def _plain_decode(s):
    c = s["case"]
    b, hkv, d = c["seqs"], c["hkv"], c["d"]
    seen = torch.arange(s["max_len"], device=DEV)[None] < s["seq_lens"][:, None]
    q = s["q"].float().view(b, hkv, c["hq"] // hkv, d)
    z = torch.matmul(q, _dense(s["k_pages"], s["k_scale"], s, seen).transpose(-1, -2)) / math.sqrt(d)
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    w = e / total
    out = torch.matmul(w, _dense(s["v_pages"], s["v_scale"], s, seen))
    got = {"out": out.reshape(b, c["hq"], d).bfloat16(),
           "lse": (m + torch.log(total)).reshape(b, c["hq"])}
    if c["scored"]:
        got["score"] = torch.where(seen[:, None], s["score_in"] + w.sum(2), s["score_out"])
    return got


def _plain_move(src, dst, s, at, ok):
    """Rows at [B, n, Hkv] of the sequences into positions 0 .. of the pages of dst_table."""
    c = s["case"]
    b, n, hkv = at.shape
    head = torch.arange(hkv, device=DEV)
    from_page = torch.gather(s["table"].long(), 1, (at // c["page"]).reshape(b, -1)).view(b, n, hkv)
    i = torch.arange(n, device=DEV)[None].expand(b, -1)
    to_page = torch.gather(s["dst_table"].long(), 1, i // c["page"])[ok]
    place = (i % c["page"])[ok]
    codes, blocks = _parts(src, c)
    to_codes, to_blocks = _parts(dst, c)
    to_codes[to_page, :, place] = codes[from_page, head, at % c["page"]][ok]
    to_blocks[to_page, :, place] = blocks[from_page, head, at % c["page"]][ok]


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
    ok = torch.arange(width, device=DEV)[None] < new[:, :, 0]
    _plain_move(s["k_pages"], s["k_dst"], s, at.permute(0, 2, 1), ok)
    _plain_move(s["v_pages"], s["v_dst"], s, at.permute(0, 2, 1), ok)
    where = _rows_of(s)
    pad = (0, budget - width)
    return {"kept": torch.nn.functional.pad(torch.where(real, kept, -1), pad, value=-1).int(),
            "new_lens": new[:, 0, 0].int(), "score": torch.nn.functional.pad(score, pad),
            "k": _plain_get(s["k_dst"], s["k_scale"], where, c),
            "v": _plain_get(s["v_dst"], s["v_scale"], where, c)}


# ------------------------------------------------------------------ the library's calls
def _desc(q, s, table, pages):
    c = s["case"]
    return q.make_paged_desc(c["seqs"], s["max_len"], pages.shape[0], c["page"], table.shape[1],
                             c["hq"], c["hkv"], c["d"], kv_fp4=True)


def _own_append(s):
    import prefill_only_cascade_gb300 as q
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"])
    q.paged_kv_append(s["desc"], s["k_new"], s["v_new"], s["start_pos"], s["table"], s["k_pages"],
                      s["v_pages"], new_offsets=s["offsets"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"])
    return _own_read(s)


def _own_read(s):
    import prefill_only_cascade_gb300 as q
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"])
    q.paged_kv_read(s["desc"], s["k_pages"], s["v_pages"], s["start_pos"], s["table"], s["k_out"],
                    s["v_out"], offsets=s["offsets"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_decode(s):
    import prefill_only_cascade_gb300 as q
    scored = s["case"]["scored"]
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"])
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


def _own_evict(s):
    import prefill_only_cascade_gb300 as q
    c = s["case"]
    if "desc" not in s:
        s["desc"] = _desc(q, s, s["table"], s["k_pages"])
        s["dst_desc"] = _desc(q, {"case": c, "max_len": min(c["budget"], s["max_len"])},
                              s["dst_table"], s["k_dst"])
        s["ws"] = torch.empty(q.paged_evict_workspace_size(s["desc"], s["k_dst"].shape[0]),
                              dtype=torch.uint8, device=DEV)
    q.paged_kv_evict(s["desc"], c["budget"], c["recent"], s["k_pages"], s["v_pages"], s["table"],
                     s["seq_lens"], s["score"], s["dst_table"], s["k_dst"], s["v_dst"], s["kept"],
                     s["new_lens"], s["ws"], score_out=s["score_out"])
    q.paged_kv_read(s["dst_desc"], s["k_dst"], s["v_dst"], s["start_pos"], s["dst_table"],
                    s["k_out"], s["v_out"], offsets=s["offsets"], k_scale=s["k_scale"],
                    v_scale=s["v_scale"])
    return {"kept": s["kept"], "new_lens": s["new_lens"], "score": s["score_out"],
            "k": s["k_out"], "v": s["v_out"]}


PLAIN = {"append": _plain_append, "read": _plain_read, "decode": _plain_decode,
         "evict": _plain_evict}
OWN = {"append": _own_append, "read": _own_read, "decode": _own_decode, "evict": _own_evict}


def run(s):
    if own:
        return OWN[s["case"]["op"]](s)
    return PLAIN[s["case"]["op"]](s)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    with torch.no_grad():
        return {"append": _exact_append, "read": _exact_read, "decode": _exact_decode,
                "evict": _exact_evict}[c["op"]](s)


def _nearest(x, least, bits, most):
    """x in 64 bits at the nearest number of `bits` bits behind the leading one, exponents from
    `least` on (below that equal steps), ties to even, at most `most` in size."""
    e = torch.frexp(x.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=least) - bits)
    return (torch.round(x / step) * step).clamp(-most, most)


def _exact_code(nibble):
    """What an e2m1 code stands for: a sign, two bits of exponent, one behind the leading one."""
    sign, e, m = nibble >> 3, (nibble >> 1) & 3, (nibble & 1).double()
    size = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e - 1))
    return torch.where(sign == 1, -size, size)


def _exact_block(byte):
    """What an e4m3 code stands for (those that are numbers)."""
    sign, e, m = byte >> 7, (byte >> 3) & 15, (byte & 7).double()
    size = torch.where(e == 0, torch.ldexp(m / 8, torch.full_like(e, -6)), torch.ldexp(1 + m / 8, e - 7))
    return torch.where(sign == 1, -size, size)


def _exact_rows(s, name, b, pos, pages=None, table="table"):
    """Rows [n, Hkv, d] of sequence b at positions pos [n] or, per head, [n, Hkv]."""
    c = s["case"]
    d, page, hkv = c["d"], c["page"], c["hkv"]
    pool = s[name + "_pages"] if pages is None else pages
    head = torch.arange(hkv, device=DEV)
    pos = pos if pos.dim() == 2 else pos[:, None].expand(-1, hkv)
    block = pool[s[table][b].long()[pos // page], head]                    # [n, Hkv, bytes]
    at = (pos % page)[..., None]
    byte = block.gather(-1, at * (d // 2) + torch.arange(d // 2, device=DEV)).int()
    code = torch.empty(*byte.shape, 2, dtype=torch.float64, device=DEV)
    code[..., 0], code[..., 1] = _exact_code(byte % 16), _exact_code(byte // 16)
    scale = block.gather(-1, page * (d // 2) + at * (d // BLOCK)
                         + torch.arange(d // BLOCK, device=DEV)).int()
    scale = _exact_block(scale) * s[name + "_scale"][b].double()[None, :, None]
    return code.reshape(*pos.shape, d) * scale.repeat_interleave(BLOCK, -1)


def _spans(s, lens):
    """(sequence, first row, first position, rows) of every sequence."""
    start, row = s["start_pos"].tolist(), 0
    for b, n in enumerate(int(x) for x in lens):
        yield b, row, start[b], n
        row += n


def _exact_append(s):
    c, got = s["case"], {}
    for name in ("k", "v"):
        x = s[name + "_new"].double()
        got[name] = torch.empty_like(x)
        for b, row, _, n in _spans(s, _lens(c)):
            one = s[name + "_scale"][b].double()[None, :, None]
            y = x[row:row + n].reshape(n, c["hkv"], -1, BLOCK)
            block = _nearest(y.abs().amax(-1) / (E2M1_MAX * one), -6, 3, E4M3_MAX) * one
            code = _nearest(y / block[..., None], 0, 1, E2M1_MAX)
            got[name][row:row + n] = torch.where(block[..., None] == 0, 0.0, code * block[..., None]) \
                .reshape(n, c["hkv"], c["d"])
    return got


def _exact_read(s):
    got = {}
    for name in ("k", "v"):
        got[name] = torch.empty(s["k_out"].shape, dtype=torch.float64, device=DEV)
        for b, row, first, n in _spans(s, _lens(s["case"])):
            got[name][row:row + n] = _exact_rows(s, name, b, first + torch.arange(n, device=DEV))
    return got


def _exact_decode(s):
    c = s["case"]
    group, hkv = c["hq"] // c["hkv"], c["hkv"]
    out = torch.zeros(c["seqs"], c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["seqs"], c["hq"], dtype=torch.float64, device=DEV)
    score = s["score_out"].double() if c["scored"] else None
    for b, n in enumerate(int(x) for x in _lens(c)):
        pos = torch.arange(n, device=DEV)
        k, v = _exact_rows(s, "k", b, pos), _exact_rows(s, "v", b, pos)
        for g in range(hkv):
            h = slice(g * group, (g + 1) * group)
            z = s["q"][b, h].double() @ k[:, g].T / math.sqrt(c["d"])
            lse[b, h] = torch.logsumexp(z, -1)
            w = torch.exp(z - lse[b, h, None])
            out[b, h] = w @ v[:, g]
            if score is not None:
                score[b, g, :n] = s["score_in"][b, g, :n].double() + w.sum(0)
    return {"out": out, "lse": lse, **({"score": score} if score is not None else {})}


def _exact_evict(s):
    c = s["case"]
    hkv, budget = c["hkv"], c["budget"]
    score = torch.zeros(c["seqs"], hkv, budget, dtype=torch.float64, device=DEV)
    host, k, v = s["score"].cpu().numpy(), [], []
    for b, n in enumerate(int(x) for x in _lens(c)):
        new = min(n, budget)
        recent = min(c["recent"], new)
        pos = np.empty((new, hkv), np.int64)
        for g in range(hkv):
            best = np.argsort(-host[b, g, :n - recent].astype(np.float64), kind="stable")[:new - recent]
            pos[:, g] = np.concatenate([np.sort(best), np.arange(n - recent, n)])
            score[b, g, :new] = torch.from_numpy(host[b, g, pos[:, g]].astype(np.float64))
        pos = torch.from_numpy(pos).to(DEV)
        k.append(_exact_rows(s, "k", b, pos))
        v.append(_exact_rows(s, "v", b, pos))
    return {"kept": None, "new_lens": None, "score": score, "k": torch.cat(k), "v": torch.cat(v)}
