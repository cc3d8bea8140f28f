"""Page calls whose requests add up past int32."""
import pytest
import torch

import canvas_rope_rotary_amd as mr
from gpu_util import say

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n_rows", [600, 1030])
def test_wants_past_int32(n_rows):
    """Requests of 2^22 pages each on a pool of 100: together past 2^31 (and 2^32).  The first is granted, those
    that want nothing are, and the small ones behind the large ones are not."""
    say("wants", n_rows)
    width = 1 << 22
    tables = torch.empty(n_rows, width, dtype=torch.int32, device="cuda")  # (only what is granted is written)
    refcount, lens = torch.zeros(100, dtype=torch.int32, device="cuda"), torch.zeros(n_rows, dtype=torch.int32, device="cuda")
    rows = list(range(n_rows))
    want = [2] + [width] * (n_rows - 3) + [0, 1]
    status = mr.pages_grow(refcount, tables, lens, i32(rows), i32(want), 1)
    assert status.tolist() == [0] + [mr.PAGES_NOT_ENOUGH] * (n_rows - 3) + [0, mr.PAGES_NOT_ENOUGH]
    assert refcount.tolist() == [1, 1] + [0] * 98
    assert lens.tolist() == [2] + [0] * (n_rows - 1)
    assert tables[0, :2].tolist() == [0, 1]
