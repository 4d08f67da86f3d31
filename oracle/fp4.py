"""Oracle for the 4-bit pages of the paged cache (numpy, CPU). Test infrastructure.

The form: blocks of 16 values of one (token, KV head) share an e4m3 scale b, a sequence's KV head
an fp32 scale S; value = e2m1(code) * b * S. OCP E2M1: a sign, two bits of exponent (bias 1), one
of mantissa, no infinities and no NaN: 0, 0.5, 1, 1.5, 2, 3, 4, 6.

Encoding rule (both sides take it in fp32): t = max|x| / (6 S), the product and the quotient
rounded; b = e4m3(t), nearest, ties to the even code, at most 448, NaN for a NaN; y = x / (b S),
the product and the quotient rounded; code = e2m1(y), nearest, ties to the even code, at most 6,
sign kept; in a block whose b is 0 or NaN all codes are 0.

A pool is [pages, Hkv, page_size * (d / 2 + d / 16)] bytes: per page and head the codes of
page_size tokens (two a byte, the even d in the low bits), then their block scales.
"""
from __future__ import annotations

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

E2M1_MAX = 6.0


def e2m1_decode(codes) -> np.ndarray:
    """Value of each E2M1 code from the OCP formula, float64."""
    c = np.asarray(codes, np.int64) & 0xF
    e, m = (c >> 1) & 3, (c & 1).astype(np.float64)
    size = np.where(e == 0, m / 2, np.ldexp(1 + m / 2, e - 1))
    return np.where(c >> 3, -size, size)


_VALUES = e2m1_decode(np.arange(8))


def e2m1_encode(x) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, saturating at 6, sign kept. No NaN."""
    x = np.asarray(x, np.float64)
    mag = np.minimum(np.abs(x), E2M1_MAX)
    off = np.abs(mag[..., None] - _VALUES)
    best = off.min(-1, keepdims=True)
    even = np.where((off == best) & (np.arange(8) % 2 == 0), 0, np.where(off == best, 1, 2))
    return (even.argmin(-1) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def quantise(rows, scale):
    """rows [T, Hkv, d] (bf16 values) under scale [Hkv] or [T, Hkv] -> codes [T, Hkv, d] and block
    scales [T, Hkv, d / 16], uint8."""
    x = np.asarray(rows, np.float32).reshape(*rows.shape[:2], rows.shape[2] // 16, 16)
    S = np.broadcast_to(np.asarray(scale, np.float32), rows.shape[:2])[..., None]
    with np.errstate(all="ignore"):
        t = np.abs(x).max(-1) / (np.float32(6) * S)
        nan = np.isnan(t)
        b = np.where(nan, 0x7F, e4m3_encode(np.where(nan, 0, t))).astype(np.uint8)
        value = e4m3_decode(b).astype(np.float32)
        y = x / (value * S)[..., None]
        dead = (nan | (value == 0))[..., None] | np.isnan(y)
        codes = np.where(dead, 0, e2m1_encode(np.where(dead, 0, y)))
    return codes.reshape(rows.shape).astype(np.uint8), b


def values(codes, blocks, scale):
    """What codes [.., Hkv, d] and blocks [.., Hkv, d / 16] stand for under scale [Hkv], float64."""
    x = e2m1_decode(codes).reshape(*codes.shape[:-1], codes.shape[-1] // 16, 16) * e4m3_decode(blocks)[..., None]
    return x.reshape(codes.shape) * np.asarray(scale, np.float64)[..., None]


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(data):
    return np.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], 2 * data.shape[-1])


def parts(pool, page, d):
    """Views [pages, Hkv, page, ..] of a pool: packed codes and block scales."""
    n, hkv, _ = pool.shape
    cut = page * d // 2
    return (pool[:, :, :cut].reshape(n, hkv, page, d // 2),
            pool[:, :, cut:].reshape(n, hkv, page, d // 16))


def join(codes, blocks):
    """A pool from packed codes [pages, Hkv, page, d / 2] and block scales [.., d / 16]."""
    return np.concatenate([codes.reshape(*codes.shape[:2], -1), blocks.reshape(*codes.shape[:2], -1)], -1)


def append(pool, page, d, new, offsets, start, table, scale):
    """The pool with rows new [T, Hkv, d] of each sequence b at start[b] .. of its pages, under
    scale [B, Hkv]; a copy."""
    codes, blocks = (x.copy() for x in parts(pool, page, d))
    for b in range(len(start)):
        c, s = quantise(new[offsets[b]:offsets[b + 1]], scale[b])
        for i in range(len(c)):
            at = start[b] + i
            codes[table[b, at // page], :, at % page] = pack(c[i])
            blocks[table[b, at // page], :, at % page] = s[i]
    return join(codes, blocks)


def rows(pool, page, d, table_row, positions, scale):
    """Rows [n, Hkv, d] at the positions of one sequence, float64."""
    codes, blocks = parts(pool, page, d)
    p = np.asarray(positions, np.int64)
    at = np.asarray(table_row, np.int64)[p // page]
    return values(unpack(codes[at, :, p % page]), blocks[at, :, p % page], scale)
