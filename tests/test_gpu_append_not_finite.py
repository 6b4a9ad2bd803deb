"""epq_pages_append of rows with infinities and NaN: the GPU packer's bytes (epq_quantize)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _packed(epq, x):
    """float32 [rows, D] -> cache rows by the packer."""
    n, D = x.shape
    b = epq.epq_quantize(epq.EPQ_Q8_0, x.view(-1, 256)).view(n, D // 32, 34)  # (the packer takes rows of 256)
    return torch.cat([b[:, :, :2].reshape(n, D // 16), b[:, :, 2:].reshape(n, D)], 1)


def _rows(D):
    """One kind of row after another: (name, row)."""
    g = torch.Generator(device="cuda").manual_seed(D)
    new = lambda: torch.randn(D, generator=g, device="cuda")  # noqa: E731
    for where in (0, 5, 31, 32, D - 1):
        for v in (math.inf, -math.inf, math.nan, 3.4e38, -3.4e38):
            x = new()
            x[where] = v
            yield x
    for first, last in ((0, 32), (32, 64), (0, D), (3, 20), (16, 48)):
        for v in (math.inf, math.nan):
            x = new()
            x[first:last] = v
            yield x
    x = new()
    x[::2], x[1::4] = math.nan, math.inf
    yield x
    yield torch.zeros(D, device="cuda")
    yield new()


@pytest.mark.parametrize("D", [128, 256])
def test_packed_bytes(epq_lib, D):
    x = torch.stack(list(_rows(D)))
    n = len(x)
    c = epq_lib.PagedKVCache(1, 1, 1, D, 1, 1, 128)
    c.table.fill_(0)
    epq_lib.epq_pages_append(x.view(1, n, D), x.flip(0).contiguous().view(1, n, D), c, 0)
    want = _packed(epq_lib, x)
    assert torch.equal(c.pool[0, 0, 0, 0, :n], want) and torch.equal(c.pool[0, 0, 0, 1, :n], want.flip(0))
    assert epq_lib.epq_device_error() == 0


def test_lone_nan(epq_lib):
    """A NaN among other numbers is code -127 under their factor; a block of nothing else has a factor of NaN."""
    x = torch.ones(1, 2, 128, device="cuda")
    x[0, 0, 5] = math.nan
    x[0, 1, 32:64] = math.nan
    c = epq_lib.PagedKVCache(1, 1, 1, 128, 1, 1, 16)
    c.table.fill_(0)
    epq_lib.epq_pages_append(x, x, c, 0)
    row = c.pool[0, 0, 0, 0, :2]
    f, codes = row[:, :8].contiguous().view(torch.float16), row[:, 8:].contiguous().view(torch.int8)
    assert torch.isfinite(f[0]).all() and codes[0, 5] == -127 and (codes[0, 6:] == 127).all()
    assert torch.isnan(f[1, 1]) and torch.isfinite(f[1, [0, 2, 3]]).all()


@pytest.mark.parametrize("rot", [20, 32, 128])
def test_position_without_angles(epq_lib, rot):
    """Appended with its rotation, such a key has factors of NaN, however little of it is turned; turned by epq_rope and
    then appended, it has them only in blocks that are turned whole, and both record the position."""
    t = epq_lib.RopeTable(rot, 4)
    x = torch.ones(1, 6, 128, device="cuda")
    for whole in (True, False):
        c = epq_lib.PagedKVCache(1, 1, 1, 128, 1, 1, 16)
        c.table.fill_(0)
        if whole:
            epq_lib.epq_pages_append(x, x, c, 0, rope=t)
        else:
            epq_lib.epq_pages_append(epq_lib.epq_rope(x, t, 1), x, c, 0)
        assert epq_lib.epq_device_error() == 6
        nan = torch.isnan(c.pool[0, 0, 0, :, :6, :8].contiguous().view(torch.float16))
        assert not nan[1].any() and not nan[0, :4].any()
        assert nan[0, 4:].sum().item() == 2 * (4 if whole else rot // 32)
