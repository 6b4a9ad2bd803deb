"""TreeDecoder.prompt refuses embeddings that its products would read as something else (on the host; nothing is launched)."""
import dataclasses

import pytest
import torch
from synthetic.workloads import DenseDecode

CFG = dataclasses.replace(DenseDecode(), layers=1, hidden=512, heads=4, kv_heads=2, inter=768, vocab=1024)


@pytest.mark.parametrize("x", [
    torch.zeros(5, 1024)[:, :512], torch.zeros(512, 5).T, torch.zeros(1, 512).expand(5, 512), torch.zeros(5, 512).half(),
    torch.zeros(5, 512, dtype=torch.float64), torch.zeros(5, 256), torch.zeros(1, 5, 512), torch.zeros(512), torch.zeros(0, 512),
], ids=lambda x: f"{list(x.shape)} {x.dtype} {x.stride()}")
def test_embeddings(epq_lib, x):
    from moe_experts_gb300 import decode

    cache = epq_lib.PagedKVCache(1, 4, CFG.kv_heads, CFG.head_dim, 1, 4, 16, "cpu")
    t = decode.TreeDecoder(CFG, epq_lib.EPQ_Q4_K, [], None, cache, 4, "cpu")
    with pytest.raises(ValueError):
        t.prompt(x, stream=0)
