"""GPU tests of attention over 4-bit pages where a warp of its own loads the tiles: what a tile's bad page
does stays with that tile's sequence and head, also for warps that have no keys in a tile."""
import pytest
import torch

import prefill_only_cascade_gb300 as q
from paged_fp4_util import Cache4, queries
from paged_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("over", [1, 33, 65])
def test_bad_tiles_among_last_tiles_with_few_keys(group, over):
    """Sequences whose last tile leaves warps without keys, each between others with a bad page in
    every tile: they are as they are without the bad ones."""
    hkv, d, page = 4, 128, 16
    lens = [2500] + [128 + over, 256 + over, 128 * 3 + over] * 40
    c = Cache4(lens, hkv, d, page, seed=over)
    hq = group * hkv
    desc, B = c.desc(hq), len(lens)
    qt = queries(over, B, hq, d)
    ws = torch.empty(q.paged_decode_workspace_size(desc), dtype=torch.uint8, device=DEV)
    bad = torch.arange(B, device=DEV) % 2 == 1
    table = torch.where(bad[:, None] & (torch.arange(c.table.shape[1], device=DEV) % 8 == 0)[None],
                        torch.full_like(c.table, c.pages), c.table)
    kw = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    q.get_device_error()
    want = torch.empty(B, hq, d, dtype=torch.bfloat16, device=DEV)
    q.paged_decode_attn(desc, qt, c.k, c.v, c.table, c.seq_lens, want, ws, **kw)
    assert q.get_device_error() == q.QUAIL_OK and torch.isfinite(want.float()).all()
    for _ in range(20):
        out = torch.full_like(want, 3.0)
        q.paged_decode_attn(desc, qt, c.k, c.v, table, c.seq_lens, out, ws, **kw)
        assert q.get_device_error() == q.QUAIL_ERR_DEVICE_BOUNDS
        assert torch.equal(out[~bad], want[~bad])
        assert torch.isnan(out[bad].float()).all()
