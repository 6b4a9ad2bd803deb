"""The readme's prompt, run as it stands on a cache in which a sequence has no room."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _prompt_lines():
    with open(README, encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    (block,) = [b for b in blocks if "epq_pages_append" in b]
    lines = block.splitlines()
    (last,) = [i for i, line in enumerate(lines) if line.startswith("epq.epq_pages_advance(")]
    return "\n".join(lines[: last + 1])


def test_prompt_without_room_for_one(epq_lib):
    """Sequence 2 is a copy of sequence 3, whose one page is partly filled; the pool has pages for sequences 0 and 1
    alone.  The shared page keeps every byte, and the copy its length."""
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = epq_lib.PagedKVCache(32, 1 + 9 + 3, 8, 128, 4, 128, 64)
    rows = torch.tensor([0, 0, 0, 40], dtype=torch.int32, device="cuda")
    assert epq_lib.epq_pages_reserve(cache, rows).tolist() == [0, 0, 0, 0]
    x = torch.randn(4, 40, 8 * 128, generator=g, device="cuda")
    for layer in range(32):
        epq_lib.epq_pages_append(x, x, cache, layer, n_tok=rows)
    epq_lib.epq_pages_advance(cache, rows)
    epq_lib.epq_pages_fork(cache, *(torch.tensor([s], dtype=torch.int32, device="cuda") for s in (3, 2)))
    page = cache.table[3, 0].item()
    before = cache.pool[:, page].clone()
    qkv = torch.randn(4, 517, (32 + 8 + 8) * 128, generator=g, device="cuda")
    exec(_prompt_lines(), {"epq": epq_lib, "torch": torch, "cache": cache, "qkv": qkv})
    assert cache.length.tolist() == [517, 129, 40, 40]
    assert cache.table[2, 0].item() == page and cache.refs[page].item() == 2
    assert torch.equal(cache.pool[:, page], before)
    assert epq_lib.epq_device_error() == 0
