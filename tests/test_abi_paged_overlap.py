"""Host-only: quail_paged_decode_attn and quail_attn_scores refuse outputs that overlap their inputs
before any launch, and nothing else on that account."""
import pytest

from test_abi_paged import BIG, INVALID, P, decode, desc, scores

ROW = 32 * 128 * 2                    # bytes of a sequence's queries
OUT = P + (1 << 24)                   # out [4, 32, 128] bf16: 32 KB
SCORES = 4 * 4 * 8 * 1000             # bytes of [4, 8, 1000] fp32


def test_the_call_is_good_otherwise():
    assert decode(desc(), out=OUT) != INVALID
    assert decode(desc(), out=OUT, si=BIG, so=BIG, stride=1000) != INVALID
    assert scores() != INVALID


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=P + 8), dict(qs=4095), dict(qs=4100), dict(kp=None), dict(vp=P + 8),
    dict(table=None), dict(lens=None), dict(lens=P + 2), dict(out=None), dict(out=OUT + 8),
    dict(lse=P + 2), dict(si=P), dict(so=P, stride=999), dict(so=P + 2, stride=1000), dict(ws=None),
    dict(ws=P + 8), dict(ws_bytes=100), dict(ks=P), dict(ks=P, vs=P),
])
def test_decode_rejects(change):
    assert decode(desc(), **{"out": OUT, **change}) == INVALID


@pytest.mark.parametrize("qs,shift,good", [
    (4096, 0, False), (4096, 16, False), (4096, -16, False), (4096, 4 * ROW - 16, False),
    (4096, 4 * ROW, True), (4096, -4 * ROW, True), (4096, -4 * ROW + 16, False),
    # rows 10 * ROW apart: out fits between two of them
    (40960, ROW, True), (40960, ROW - 16, False), (40960, 6 * ROW, True), (40960, 6 * ROW + 16, False),
    (40960, 31 * ROW, True), (40960, 31 * ROW - 16, False), (40960, 24 * ROW, True),
    (40960, 29 * ROW, False), (40960, -4 * ROW, True), (40960, -4 * ROW + 16, False),
])
def test_out_over_the_queries(qs, shift, good):
    assert (decode(desc(), q=BIG, qs=qs, out=BIG + shift) != INVALID) == good


@pytest.mark.parametrize("shift,good", [(0, True), (4, False), (-4, False), (SCORES - 4, False),
                                        (4 - SCORES, False), (SCORES, True), (-SCORES, True)])
def test_scores_that_partly_overlap(shift, good):
    assert (decode(desc(), out=OUT, si=BIG, so=BIG + shift, stride=1000) != INVALID) == good
    n = 4 * 2 * 2 * 40
    if abs(shift) > 4:
        shift += (n - SCORES) * (1 if shift > 0 else -1)
    assert (scores(si=BIG, so=BIG + shift) != INVALID) == good


def test_nothing_to_overlap():
    assert decode(desc(num_seqs=0), q=P, out=P) != INVALID
    assert scores(seqs=0, tq=0, tk=0, si=P, so=P + 4) != INVALID
