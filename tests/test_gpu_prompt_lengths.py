"""epq_attention_prompt on lengths that no sequence of the cache can have: below 0 as 0, past the table as its end."""
import pytest
import torch
from test_gpu_prompt_attention import Case, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [0, 16])
def test_below_zero(epq_lib, window, D):
    c = Case(epq_lib, [0, 30], [70, 40], 4, 2, D, 16, window=window, seed=33)
    want = c.check()
    c.c.length[0] = -5
    assert torch.equal(c.run(), want)
    c.c.length[0] = -2**31
    assert torch.equal(c.run(), want)
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("length", [2**31 - 1, 176])
def test_past_the_table(epq_lib, length, D):
    """Ten pages of 16 in a table of eleven: every token sees the 160 positions that have a page, and the others are
    recorded; with a window it sees none.  Bounds as in test_gpu_prompt_accuracy."""
    T, t, G = 160, 64, 2
    c = Case(epq_lib, [96, 5], [t, 40], 4, 2, D, 16, seed=35)
    assert c.c.max_pages == 11
    other = c.check()[1]
    c.c.length[0] = length
    out = c.run()
    assert epq_lib.epq_device_error() == 5
    assert torch.equal(out[1], other)
    x = _values(c.rows(0))
    for h in range(2):
        K, V = x[:, h, 0], x[:, h, 1]
        q = c.q[0, :t].view(t, 4, D)[:, h * G:(h + 1) * G].double()
        w = torch.softmax(q @ K.T * c.scale, -1)
        ds = (32 + D / 4) * 2.0 ** -24 * (q.abs() @ K.abs().T * c.scale).amax(-1, keepdim=True)
        bound = (w @ V.abs()) * (torch.expm1(2 * ds) + (128 + T * D / 2048) * 2.0 ** -24) + 2.0 ** -39 * V.abs().sum(0)
        assert ((out[0].view(t, 4, D)[:, h * G:(h + 1) * G].double() - w @ V).abs() <= bound).all()
    c.window = 16
    assert not c.run()[0].any()
    assert epq_lib.epq_device_error() == 5
