"""TreeDecoder.prompt captured in a graph: a chunk of a prompt replayed with other embeddings, behind itself."""
import pytest
import torch
from test_gpu_prompt_decode import _decoder, setup  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 21])
def test_prompt_captured(epq_lib, cuda_dev, setup, n):  # noqa: F811
    a, b = _decoder(epq_lib, cuda_dev, setup, 4), _decoder(epq_lib, cuda_dev, setup, 4)
    x = setup[3][:n].clone()
    b.prompt(x)  # (what a first call sets up)
    epq_lib.epq_pages_truncate(b.cache, torch.zeros(1, dtype=torch.int32, device=cuda_dev))
    b.cache.pool.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = b.prompt(x)
    room = 24 * 16 // n
    for k in range(min(room, 20)):
        x.copy_(setup[3][n * k % 900:][:n])
        want = a.prompt(x)
        graph.replay()
        assert torch.equal(got, want) and a.status.item() == b.status.item() == 0
        assert torch.equal(a.cache.pool, b.cache.pool) and torch.equal(a.cache.length, b.cache.length)
    if n > 1:  # no room: nothing changes
        while b.status.item() == 0:
            graph.replay()
        length = b.cache.length.item()
        before = b.cache.pool.clone()
        graph.replay()
        assert b.cache.length.item() == length and torch.equal(b.cache.pool, before)
    assert epq_lib.epq_device_error() == 0
