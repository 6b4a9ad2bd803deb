"""Refusals of epq_attention_prompt, found on the host before the device is
looked at (tensors here live on the CPU and are never read)."""
import ctypes
import math

import pytest
import torch

EPQ_ERR_ARG, EPQ_ERR_SHAPE, EPQ_ERR_ALIGN, EPQ_ERR_WORKSPACE = 1, 3, 4, 5


def _cache(epq):
    return epq.PagedKVCache(2, 6, 2, 128, 3, 4, 16, "cpu")


def _call(epq, ntok=5, heads=4, layer=0, scale=0.1, q=None, **kw):
    return epq.epq_attention_prompt(torch.zeros(3, ntok, heads * 128) if q is None else q, _cache(epq), layer, heads, scale, stream=0, **kw)


@pytest.mark.parametrize("status, kw", [
    (EPQ_ERR_ARG, dict(layer=2)), (EPQ_ERR_ARG, dict(layer=-1)), (EPQ_ERR_ARG, dict(scale=0.0)), (EPQ_ERR_ARG, dict(scale=-1.0)),
    (EPQ_ERR_ARG, dict(scale=math.inf)), (EPQ_ERR_ARG, dict(scale=math.nan)), (EPQ_ERR_ARG, dict(window=-1)),
    (EPQ_ERR_WORKSPACE, dict(workspace=torch.zeros(0, dtype=torch.uint8))), (EPQ_ERR_ALIGN, dict(q=torch.zeros(3, 5, 514)[..., 2:])),
    (EPQ_ERR_ALIGN, dict(q=torch.zeros(3 * 5 * 512 + 1)[1:].view(3, 5, 512))),
])
def test_status(epq_lib, status, kw):
    with pytest.raises(epq_lib.EpqError) as e:
        _call(epq_lib, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(heads=3), dict(heads=34), dict(ntok=0), dict(q=torch.zeros(3, 640)), dict(q=torch.zeros(2, 5, 512)), dict(q=torch.zeros(3, 5, 512).half()),
    dict(q=torch.zeros(3, 5, 1024)[..., ::2]), dict(q=torch.zeros(1, 5, 512).expand(3, 5, 512)), dict(n_tok=torch.zeros(3)),
    dict(n_tok=torch.zeros(2, dtype=torch.int32)), dict(out=torch.zeros(3, 5, 1024)[..., :512]),
])
def test_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _call(epq_lib, **kw)


def test_workspace_and_sizes(epq_lib):
    lib, c = epq_lib.load(), _cache(epq_lib)
    size = lambda heads, ntok: lib.epq_attention_prompt_workspace_bytes(ctypes.byref(c._p), heads, ntok)  # noqa: E731
    assert size(4, 1) > 0 and size(4, 5000) > 0 and size(32, 5) > 0
    assert size(3, 5) == 0 and size(34, 5) == 0 and size(4, 0) == 0 and size(0, 5) == 0 and size(4, 1 << 24) == 0
    q = torch.zeros(3, 5, 512)
    w = torch.zeros(size(4, 5) + 16, dtype=torch.uint8)
    call = lambda **kw: lib.epq_attention_prompt(ctypes.byref(c._p), 0, *[kw.get(k, d) for k, d in (  # noqa: E731
        ("q", q.data_ptr()), ("heads", 4), ("ntok", 5), ("scale", 0.1), ("o", None), ("out", q.data_ptr()), ("ws", w.data_ptr()), ("n", size(4, 5)))], None)
    assert call(q=None) == EPQ_ERR_ARG and call(out=None) == EPQ_ERR_ARG and call(ws=None) == EPQ_ERR_WORKSPACE
    assert call(n=size(4, 5) - 1) == EPQ_ERR_WORKSPACE and call(ws=w.data_ptr() + 8) == EPQ_ERR_ALIGN
    assert call(heads=5) == EPQ_ERR_SHAPE and call(ntok=0) == EPQ_ERR_SHAPE
    O = epq_lib._lib.PromptOpts
    assert call(o=ctypes.byref(O(q_ld=514))) == EPQ_ERR_ALIGN and call(o=ctypes.byref(O(q_ld=-512))) == EPQ_ERR_ARG
