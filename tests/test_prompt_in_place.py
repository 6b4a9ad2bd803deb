"""epq_attention_prompt with its output over its queries: refused where an item would read another's output."""
import ctypes

import pytest
import torch

EPQ_ERR_ARG = 1


@pytest.mark.parametrize("D, strides", [(256, {}), (128, dict(q_ld=1024)), (128, dict(q_seq_ld=512)), (256, dict(q_ld=1024))])
def test_refused(epq_lib, D, strides):
    lib = epq_lib.load()
    c = epq_lib.PagedKVCache(1, 6, 2, D, 3, 4, 16, "cpu")
    ws = epq_lib.epq_attention_prompt_workspace(c, 4, 5)
    q = torch.zeros(3 * 5 * 4 * D * 2)
    o = epq_lib._lib.PromptOpts(**strides)
    st = lib.epq_attention_prompt(ctypes.byref(c._p), 0, q.data_ptr(), 4, 5, 0.1, ctypes.byref(o), q.data_ptr(), ws.data_ptr(),
                                  ws.numel(), None)
    assert st == EPQ_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [
    ([0], [65], 32, 8, 128, 64, 0), ([0, 333, 401, 5], [200, 129, 1, 0], 16, 16, 128, 16, 0), ([31, 32], [33, 96], 16, 1, 128, 16, 0),
    ([0, 2000], [700, 130], 6, 2, 128, 64, 64), ([20000, 0, 17], [1, 1, 1], 32, 8, 128, 64, 0),
    ([i % 7 * 3 for i in range(256)], [20 + i % 3 for i in range(256)], 16, 1, 128, 16, 0),
])
def test_heads_of_128(epq_lib, shape):
    from test_gpu_prompt_attention import Case

    c = Case(epq_lib, *shape)
    want = c.run()
    for _ in range(5):
        q = c.q.clone()
        assert c.run(q=q, out=q) is q and torch.equal(q, want)


@pytest.mark.gpu
def test_heads_of_256(epq_lib):
    from test_gpu_prompt_attention import Case

    c = Case(epq_lib, [7], [50], 15, 3, 256, 64)
    with pytest.raises(epq_lib.EpqError) as e:
        c.run(out=c.q)
    assert e.value.status == EPQ_ERR_ARG
