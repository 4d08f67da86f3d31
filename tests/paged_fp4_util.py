"""Inputs and error bounds of the tests of 4-bit pages."""
import math

import numpy as np
import torch

import prefill_only_cascade_gb300 as q
from oracle import fp4, paged
from paged_util import BF16, DEV, U32, block_table, f64


class Cache4:
    """Random codes (all sixteen) and block scales for sequences of the given lengths; what no
    sequence holds has block scales that are NaN."""

    def __init__(self, lens, hkv, d, page, seed=0, width=None, blocks=(0x20, 0x78)):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.hkv, self.d = [int(n) for n in lens], page, hkv, d
        self.table_np, self.pages = block_table(lens, page, rng, width)
        held = np.zeros(self.pages * page, bool)
        for b, n in enumerate(self.lens):
            held[paged.slots(self.table_np[b], np.arange(n), page)] = True
        held = held.reshape(self.pages, 1, page, 1)
        pools = []
        for _ in range(2):
            codes = rng.integers(0, 256, (self.pages, hkv, page, d // 2), dtype=np.uint8)
            scales = rng.integers(blocks[0], blocks[1] + 1, (self.pages, hkv, page, d // 16)).astype(np.uint8)
            pools.append(fp4.join(codes, np.where(held, scales, np.uint8(0x7F))))
        self.k_np, self.v_np = pools
        self.k, self.v = (torch.from_numpy(x).to(DEV) for x in pools)
        # values of size about one: block scales are up to 256, codes up to 6
        self.ks_np, self.vs_np = ((0.5 + rng.random((len(lens), hkv))).astype(np.float32) / 300
                                  for _ in range(2))
        self.k_scale, self.v_scale = (torch.from_numpy(x).to(DEV) for x in (self.ks_np, self.vs_np))
        self.table = torch.from_numpy(self.table_np).to(DEV)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def rows(self, b, positions=None):
        """K and V [n, Hkv, d] of sequence b in 64 bits."""
        at = np.arange(self.lens[b]) if positions is None else positions
        return tuple(fp4.rows(pool, self.page, self.d, self.table_np[b], at, scale[b])
                     for pool, scale in ((self.k_np, self.ks_np), (self.v_np, self.vs_np)))

    def desc(self, hq, max_len=None, scale=0.0):
        return q.make_paged_desc(len(self.lens), max(self.lens) if max_len is None else max_len,
                                 self.pages, self.page, self.table.shape[1], hq, self.hkv, self.d,
                                 scale, kv_fp4=True)


def decode_bounds(qh, k, v, scale):
    """Error bounds of one sequence: out [Hq, d] (before its rounding to bf16), lse [Hq], and the
    relative error of a weight [Hq].

    Codes times block scales are exact in f16, Q is exact but for bits below 2^-38 of the head's
    largest. A score in log2 units is a sum of d exact products in fp32 (error (d + 2) u of the
    sum of magnitudes X), scaled by three rounded factors (4 u) and reduced by the maximum (u each
    of two values of at most X); exp2 adds 2^-22. P is the sum of two f16 (2^-22, and its floor
    2^-38 of the largest weight for each key, of the sequence's sum at most once the largest is
    part of it); sums of n terms add n u, join, scale and quotient a few u more."""
    n, hkv, d = k.shape
    group = qh.shape[0] // hkv
    X = scale * math.log2(math.e) * np.array(
        [np.max(np.abs(k[:, h // group]) @ np.abs(qh[h])) for h in range(qh.shape[0])])
    err_x = (d + 8) * U32 * X
    weight = 2 * (math.log(2) * err_x + 2.0 ** -22) + (n + 16) * U32
    absv, _, _ = paged.decode(qh, k, np.abs(v), scale)
    # the floor is absolute: 2^-38 of the largest weight (at most 1), times every |v|
    floor = 2.0 ** -38 * np.stack([np.abs(v[:, h // group]).sum(0) for h in range(qh.shape[0])])
    out = (weight + 2.0 ** -21 + n * U32)[:, None] * absv + floor
    lse = math.log(2) * (2 * err_x + 4 * X * U32) + (n + 16) * U32 + 2.0 ** -20
    return out, lse, weight + 2 * lse


def run_decode(cache, qt, hq, scored=False, score_in=None, max_len=None, scale=0.0, k=None, v=None):
    desc = cache.desc(hq, max_len, scale)
    B = len(cache.lens)
    ws = torch.full((max(q.paged_decode_workspace_size(desc, scored), 16),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    out = torch.full((B, hq, cache.d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, hq), 3.0, device=DEV)
    score_out = None
    if scored:
        score_out = torch.full((B, cache.hkv, max(desc.max_seq_len, 1) + 5), -3.0, device=DEV)
    q.paged_decode_attn(desc, qt, cache.k if k is None else k, cache.v if v is None else v, cache.table,
                        cache.seq_lens, out, ws, lse=lse, k_scale=cache.k_scale, v_scale=cache.v_scale,
                        score_in=score_in, score_out=score_out)
    return out, lse, score_out


def check_decode(cache, qt, hq, out, lse, score=None, score_in=None, scale=0.0, only=None):
    scale = scale or 1 / math.sqrt(cache.d)
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
            t_out, t_lse, t_w = decode_bounds(q64[b], k, v, scale)
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


def queries(seed, *shape, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).bfloat16().to(DEV)
