"""Pins of oracle/fp4.py: the E2M1 table, ties, round trips, brute force and error bounds."""
import numpy as np
import pytest
import torch

from oracle import fp4
from oracle.fp8 import e4m3_decode


def test_e2m1_table():
    want = [0, .5, 1, 1.5, 2, 3, 4, 6]
    np.testing.assert_array_equal(fp4.e2m1_decode(np.arange(16)), want + [-x for x in want])
    codes = np.arange(16)
    np.testing.assert_array_equal(fp4.e2m1_encode(fp4.e2m1_decode(codes)), codes)


def test_ties_go_to_the_even_code_and_large_values_saturate():
    x = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.0001, 7.0, np.inf, -0.25, -0.0, -5.0]
    np.testing.assert_array_equal(fp4.e2m1_encode(x), [0, 2, 2, 4, 4, 6, 6, 7, 7, 7, 8, 8, 14])


def test_encode_is_the_nearest_value():
    x = np.random.default_rng(0).uniform(-7, 7, 4000)
    got = fp4.e2m1_decode(fp4.e2m1_encode(x))
    grid = fp4.e2m1_decode(np.arange(16))
    np.testing.assert_array_equal(np.abs(got - x), np.abs(grid[None] - x[:, None]).min(1))


def test_quantise_error_and_block_scale():
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(40, 3, 64))).bfloat16().float().numpy()
    scale = np.abs(x).max((0, 2)).astype(np.float32) / np.float32(2688)
    codes, blocks = fp4.quantise(x, scale)
    got = fp4.values(codes, blocks, scale)
    b = e4m3_decode(blocks) * scale[None, :, None].astype(np.float64)
    amax = np.abs(x).reshape(40, 3, 4, 16).max(-1)
    assert (np.abs(b - amax / 6) <= amax / 6 * 2.0 ** -4 * 1.001).all()   # half a step of e4m3
    # half of the widest gap (1 between 4 and 6), and 6 b may lie a half step of e4m3 below amax
    assert (np.abs(got - x).reshape(40, 3, 4, 16).max(-1) <= np.maximum(b, amax - 6 * b) * 1.001).all()


def test_quantise_one_block_by_hand():
    x = np.array([6, -3, 2.5, 0.5, 0.25, 5, 1.75, 0, -0.75, 6, 4, 3.5, 1, 1.25, -6, 0.2],
                 np.float32)[None, None]
    codes, blocks = fp4.quantise(x, [np.float32(1 / 16)])
    assert e4m3_decode(blocks)[0, 0, 0] == 16
    np.testing.assert_array_equal(fp4.values(codes, blocks, [1 / 16])[0, 0],
                                  [6, -3, 2, .5, 0, 4, 2, 0, -1, 6, 4, 4, 1, 1, -6, 0])


@pytest.mark.parametrize("what,block,code", [
    (np.zeros(16), 0.0, 0), (np.full(16, 1e-30), 0.0, 0), (np.full(16, np.nan), np.nan, 0),
    (np.r_[np.nan, np.ones(15)], np.nan, 0), (np.r_[np.inf, np.ones(15)], 448.0, None)])
def test_quantise_corners(what, block, code):
    codes, blocks = fp4.quantise(what[None, None].astype(np.float32), [np.float32(0.01)])
    np.testing.assert_array_equal(e4m3_decode(blocks).ravel(), [block])
    if code is not None:
        assert (codes == code).all()
    else:
        assert codes[0, 0, 0] == 7


def test_append_then_rows():
    rng = np.random.default_rng(2)
    new = rng.normal(size=(9, 2, 64)).astype(np.float32)
    scale = np.full((2, 2), 0.002, np.float32)
    table = np.array([[3, 1], [0, 2]])
    pool = np.full((4, 2, 16 * 36), 0x7F, np.uint8)
    got = fp4.append(pool, 16, 64, new, [0, 4, 9], [14, 0], table, scale)
    assert (got[2] == 0x7F).all()
    for b, lo, hi, first in ((0, 0, 4, 14), (1, 4, 9, 0)):
        c, s = fp4.quantise(new[lo:hi], scale[b])
        np.testing.assert_array_equal(
            fp4.rows(got, 16, 64, table[b], first + np.arange(hi - lo), scale[b]),
            fp4.values(c, s, scale[b]))
    codes, blocks = fp4.parts(got, 16, 64)
    np.testing.assert_array_equal(fp4.pack(fp4.unpack(codes)), codes)
    np.testing.assert_array_equal(fp4.join(codes, blocks), got)
