"""Refusals of epq_logits_adjust, found on the host before the device is looked
at (tensors here live on the CPU and are never read)."""
import ctypes

import pytest
import torch

EPQ_ERR_ARG, EPQ_ERR_SHAPE, EPQ_ERR_ALIGN = 1, 3, 4


def _adjust(epq, nseq=2, ntok=3, vocab=40, logits=None, **kw):
    return epq.epq_logits_adjust(torch.zeros(nseq, ntok, vocab) if logits is None else logits, stream=0, **kw)


@pytest.mark.parametrize("kw", [
    dict(logits=torch.zeros(3, 40)), dict(logits=torch.zeros(2, 3, 40, dtype=torch.float16)),
    dict(logits=torch.zeros(2, 3, 80)[..., :40]), dict(penalties=torch.zeros(2, 2)), dict(penalties=torch.zeros(3, 3)),
    dict(history=torch.zeros(5, dtype=torch.int32)), dict(history=torch.zeros(3, 5, dtype=torch.int32)),
    dict(history=torch.zeros(2, 5)), dict(history_len=torch.zeros(3, dtype=torch.int32)),
    dict(prompt_len=torch.zeros(2)), dict(tokens=torch.zeros(2, 4, dtype=torch.int32)),
    dict(mask=torch.zeros(2, 3, dtype=torch.int32)), dict(n_tok=torch.zeros(1, dtype=torch.int32)),
    dict(bias=torch.zeros(2, 4)), dict(bias_ids=torch.zeros(2, 4, dtype=torch.int32)),
    dict(bias_ids=torch.zeros(2, 4, dtype=torch.int32), bias=torch.zeros(2, 5)),
    dict(bias_ids=torch.zeros(4, dtype=torch.int32), bias=torch.zeros(4)),
    dict(allowed=torch.zeros(2, 3, 1, dtype=torch.int32)), dict(allowed=torch.zeros(2, 3, 40, dtype=torch.bool)),
    dict(out=torch.zeros(2, 3, 41)),
])
def test_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _adjust(epq_lib, **kw)


def test_status(epq_lib):
    for kw in (dict(ntok=65, tokens=torch.zeros(2, 65, dtype=torch.int32)),):
        with pytest.raises(epq_lib.EpqError) as e:
            _adjust(epq_lib, **kw)
        assert e.value.status == EPQ_ERR_SHAPE
    with pytest.raises(epq_lib.EpqError) as e:
        _adjust(epq_lib, ntok=0)  # a tensor of nothing has no address
    assert e.value.status == EPQ_ERR_ARG


def test_c_status(epq_lib):
    """What the binding cannot pass."""
    lib, O = epq_lib.load(), epq_lib._lib.LogitsOpts
    x = torch.zeros(1 << 10)
    a = x.data_ptr()
    call = lambda o=O(), x=a, y=a, v=40, n=2, t=3: lib.epq_logits_adjust(x, v, n, t, ctypes.byref(o), y, None)  # noqa: E731
    assert call(x=None) == EPQ_ERR_ARG and call(y=None) == EPQ_ERR_ARG
    assert call(v=0) == EPQ_ERR_SHAPE and call(v=(1 << 24) + 1) == EPQ_ERR_SHAPE and call(n=0) == EPQ_ERR_SHAPE
    assert call(t=0) == EPQ_ERR_SHAPE and call(n=1 << 12, t=1 << 12) == EPQ_ERR_SHAPE
    assert call(o=O(max_history=5)) == EPQ_ERR_ARG and call(o=O(max_history=-1)) == EPQ_ERR_SHAPE
    assert call(o=O(n_bias=1, bias=a)) == EPQ_ERR_ARG and call(o=O(n_bias=1, bias_ids=a)) == EPQ_ERR_ARG
    assert call(o=O(n_bias=-1)) == EPQ_ERR_SHAPE
    assert call(o=O(ld=39)) == EPQ_ERR_ARG and call(o=O(out_ld=-40)) == EPQ_ERR_ARG
    assert call(o=O(ld=48)) == EPQ_ERR_ARG  # in place with another stride
    assert call(x=a + 2) == EPQ_ERR_ALIGN and call(o=O(mask=a + 4)) == EPQ_ERR_ALIGN
    assert call(o=O(n_tok=a + 1)) == EPQ_ERR_ALIGN
