"""Inputs, reference results and error bounds of the paged-cache tests."""
import math

import numpy as np
import torch

import prefill_only_cascade_gb300 as q
from oracle import paged

U32 = 2.0 ** -24                        # half a step of fp32
BF16 = 2.0 ** -8                        # half a step of bf16
DEV = "cuda"


def f64(x):
    return x.detach().to("cpu", torch.float64).numpy()


def block_table(lens, page, rng, width=None, spare=3):
    """Pages in a random order; entries past a sequence's last page name no page."""
    need = [-(-int(n) // page) for n in lens]
    total = sum(need) + spare
    order = rng.permutation(total)
    width = max(max(need, default=0), 1) if width is None else width
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, total


class Cache:
    """Random pages for sequences of the given lengths. Everything that no sequence holds is
    NaN. Codes come with scales near 1 / 90."""

    def __init__(self, lens, hkv, d, page, fp8, seed=0, width=None):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.fp8 = [int(n) for n in lens], page, fp8
        self.table_np, self.pages = block_table(lens, page, rng, width)
        shape = (self.pages, page, hkv, d)
        self.k_scale = self.v_scale = None
        gen = torch.Generator().manual_seed(seed)
        pool = []
        for _ in range(2):
            x = torch.randn(shape, generator=gen)
            held = torch.zeros(self.pages * page, dtype=torch.bool)
            for b, n in enumerate(self.lens):
                held[torch.from_numpy(paged.slots(self.table_np[b], np.arange(n), page))] = True
            held = held.view(self.pages, page, 1, 1)
            if fp8:
                x = (x * 90).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                x = torch.where(held, x, torch.full_like(x, 0x7F)).view(torch.float8_e4m3fn)
            else:
                x = torch.where(held, x, torch.full_like(x, math.nan)).bfloat16()
            pool.append(x)
        self.k, self.v = (x.to(DEV) for x in pool)
        self.k64, self.v64 = (x.to(torch.float64).numpy().reshape(-1, hkv, d) for x in pool)
        if fp8:
            self.k_scale, self.v_scale = ((0.5 + torch.rand(len(lens), hkv, generator=gen)) / 90
                                          for _ in range(2))
            self.ks64, self.vs64 = f64(self.k_scale), f64(self.v_scale)
            self.k_scale, self.v_scale = self.k_scale.to(DEV), self.v_scale.to(DEV)
        self.table = torch.from_numpy(self.table_np).to(DEV)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def rows(self, b):
        """K and V [n, Hkv, d] of sequence b in 64 bits."""
        at = paged.slots(self.table_np[b], np.arange(self.lens[b]), self.page)
        k, v = self.k64[at], self.v64[at]
        if self.fp8:
            k, v = k * self.ks64[b][None, :, None], v * self.vs64[b][None, :, None]
        return k, v

    def desc(self, hq, max_len=None, scale=0.0):
        return q.make_paged_desc(len(self.lens), max(self.lens) if max_len is None else max_len,
                                 self.pages, self.page, self.table.shape[1], hq, self.k.shape[2],
                                 self.k.shape[3], scale, self.fp8)


def decode_bounds(qh, k, v, scale, fp8):
    """Error bounds of one sequence: out [Hq, d] (before its rounding to bf16), lse [Hq], and the
    relative error of a weight [Hq].

    A score in log2 units is a sum of d exact products in fp32 (error (d + 2) u of the sum of
    magnitudes X), scaled by a rounded factor (2 u) and reduced by the maximum (u each of two
    values of at most X); exp2 adds 2^-22. The weights are sums' quotients: the sum of n terms
    adds n u and the join and the final quotient a few u more, P = hi + lo 2^-17 (bf16) or one
    f16 rounding 2^-11 with its floor 2^-38 of the largest (e4m3)."""
    n, hkv, d = k.shape
    group = qh.shape[0] // hkv
    X = scale * math.log2(math.e) * np.array(
        [np.max(np.abs(k[:, h // group]) @ np.abs(qh[h])) for h in range(qh.shape[0])])
    err_x = (d + 6) * U32 * X
    weight = 2 * (math.log(2) * err_x + 2.0 ** -22) + (n + 16) * U32
    p_err = 2.0 ** -11 + n * 2.0 ** -38 if fp8 else 2.0 ** -16
    absv = np.stack([paged.decode(qh, k, np.abs(v), scale)[0][h] for h in range(qh.shape[0])])
    out = (weight + p_err + n * U32)[:, None] * absv
    lse = math.log(2) * (2 * err_x + 4 * X * U32) + (n + 16) * U32 + 2.0 ** -20
    return out, lse, weight + 2 * lse


def run_decode(cache, qt, hq, scored=False, score_in=None, max_len=None, scale=0.0, out=None,
               score_out=None):
    desc = cache.desc(hq, max_len, scale)
    B, d = len(cache.lens), cache.k.shape[3]
    ws = torch.full((max(q.paged_decode_workspace_size(desc, scored), 16),), 0xA5,
                    dtype=torch.uint8, device=DEV)
    out = torch.full((B, hq, d), 3.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    lse = torch.full((B, hq), 3.0, device=DEV)
    if scored and score_out is None:
        score_out = torch.full((B, cache.k.shape[2], max(desc.max_seq_len, 1) + 5), -3.0, device=DEV)
    q.paged_decode_attn(desc, qt, cache.k, cache.v, cache.table, cache.seq_lens, out, ws, lse=lse,
                        k_scale=cache.k_scale, v_scale=cache.v_scale, score_in=score_in,
                        score_out=score_out)
    return out, lse, score_out


def check_decode(cache, qt, hq, out, lse, score=None, score_in=None, scale=0.0, only=None):
    d = qt.shape[2]
    scale = scale or 1 / math.sqrt(d)
    o, l_, q64 = f64(out), f64(lse), f64(qt)
    sc = None if score is None else f64(score)
    for b, n in enumerate(cache.lens):
        if only is not None and b not in only:
            continue
        if n == 0:
            assert (o[b] == 0).all() and (l_[b] == -np.inf).all()
        else:
            k, v = cache.rows(b)
            ref, ref_lse, w = paged.decode(q64[b], k, v, scale)
            t_out, t_lse, t_w = decode_bounds(q64[b], k, v, scale, cache.fp8)
            assert np.isfinite(o[b]).all(), b
            assert (np.abs(o[b] - ref) <= t_out + BF16 * (np.abs(ref) + t_out) + 1e-38).all(), \
                (b, np.abs(o[b] - ref).max(), t_out.max())
            assert (np.abs(l_[b] - ref_lse) <= t_lse).all(), (b, np.abs(l_[b] - ref_lse).max())
            if sc is not None:
                base = 0.0 if score_in is None else f64(score_in)[b][:, :n]
                tol = t_w.max() * w + 4 * U32 * (np.abs(base) + w) + 1e-37
                assert (np.abs(sc[b][:, :n] - base - w) <= tol).all(), b
        if sc is not None:
            assert (sc[b][:, n:] == -3.0).all()      # behind the sequence: as it was
