"""The paged calls' native argument checks on a host without a GPU: None to everything, whatever it is,
and no error left behind."""
import pytest
import torch

import prefill_only_cascade_gb300 as q

pytestmark = pytest.mark.skipif(q._calls is None, reason="built without PyTorch's or Python's headers")
DESC = q.make_paged_desc(2, 30, 8, 16, 2, 4, 2, 64, kv_fp4=True)
COUNTS = {"append": 10, "read": 10, "decode": 13, "evict": 15}


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("desc", [DESC, None, 3, b"x" * 40, torch.zeros(40)])
def test_nothing_but_none(name, desc):
    call, n = getattr(q._calls, name), COUNTS[name] - 1
    for x in (None, 3, -2 ** 70, "x", torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32),
              torch.zeros(3, 2).to_sparse(), torch.nn.Parameter(torch.zeros(2, 2, 64, dtype=torch.bfloat16))):
        assert call(desc, *[x] * n) is None
    assert call() is None and call(desc) is None and call(desc, *[1] * (n + 1)) is None


def test_bind_refuses():
    for args in ((), (1,) * 5, (q.PagedDesc, 0, 1, 1, 1), (q.PagedDesc, "x", 1, 1, 1)):
        with pytest.raises((TypeError, ValueError)):
            q._calls.bind(*args)
