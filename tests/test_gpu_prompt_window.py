"""What lies below a window of epq_attention_prompt is as if it were not there: pages that are gone, factors that
are not finite, factors that would set a tile's scale."""
import math

import pytest
import torch
from test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


def _case(epq, D, P):
    # the first tile of each row tile begins below the oldest position that any of its tokens sees
    return Case(epq, [250, 1000, 40, 1023], [1, 150, 3, 40], 4, 2, D, P, window=16, seed=25)


def _below(c, s):
    """Positions of a sequence that none of its tokens sees."""
    return max(c.lengths[s] - c.window + 1, 0)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_pages_below_the_window_are_not_missed(epq_lib, D, P):
    """A page that no token sees may be gone: the same output, and nothing is recorded."""
    c = _case(epq_lib, D, P)
    want = c.check()
    assert epq_lib.epq_device_error() == 0
    gone = [_below(c, s) // P for s in range(len(c.lengths))]
    tile = 128 if D == 128 else 64
    assert P >= tile or any(n * P % tile for n in gone)  # a tile is gone in part
    for s, n in enumerate(gone):
        c.c.table[s, :n] = -1
    assert torch.equal(c.run(), want)
    assert epq_lib.epq_device_error() == 0
    c.c.table[0, gone[0]] = -1  # the first page that is seen
    c.run()
    assert epq_lib.epq_device_error() == 5


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("factor", [math.nan, math.inf, 65504.0, 0.0])
def test_rows_below_the_window_change_nothing(epq_lib, D, factor):
    c = _case(epq_lib, D, 64)
    want = c.check()
    for s in range(len(c.lengths)):
        pos = torch.arange(_below(c, s), device="cuda")
        rows = c.rows(s)[: len(pos)].clone()
        rows[..., : D // 16].view(torch.float16)[:] = factor
        c.put(s, pos, rows)
    assert torch.equal(c.run(), want)
    assert epq_lib.epq_device_error() == 0
