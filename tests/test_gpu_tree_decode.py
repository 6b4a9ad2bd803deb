"""The verification step of a small dense decoder (TreeDecoder) against the
one-token decode path: a chain of drafted tokens must give the logits that
decoding them one after the other gives, a tree those of each of its paths,
and a committed step must leave the cache as if its accepted tokens had been
decoded."""
import dataclasses
import math

import pytest
import torch

import synthetic
from synthetic.workloads import DenseDecode

pytestmark = pytest.mark.gpu

CFG = dataclasses.replace(DenseDecode(), layers=2, hidden=512, heads=4, kv_heads=2, inter=768, vocab=1024)
CTX, NTOK = 75, 6


@pytest.fixture(scope="module")
def setup(epq_lib, cuda_dev):
    from moe_experts_gb300 import decode

    H, rows = CFG.hidden, CFG.q_rows + 2 * CFG.kv_rows
    pack = lambda r, c, seed: epq_lib.epq_quantize(epq_lib.EPQ_Q4_K, synthetic.student_t((r, c), seed=seed, scale=0.05).to(cuda_dev))  # noqa: E731
    layers = [(pack(rows, H, 10 * i), pack(H, CFG.q_rows, 10 * i + 1), pack(2 * CFG.inter, H, 10 * i + 2), pack(H, CFG.inter, 10 * i + 3))
              for i in range(CFG.layers)]
    head = pack(CFG.vocab, H, 99)
    x = synthetic.normal((NTOK, H), seed=5).to(cuda_dev)
    return decode, layers, head, x


def _one_by_one(epq, dev, setup, order, monkeypatch):
    """Logits of the tokens `order` decoded one after the other, and the caches."""
    decode, layers, head, x = setup
    monkeypatch.setattr(decode, "SKIP_LOG", -math.inf)  # the tree attention keeps every position
    d = decode.DenseDecoder(CFG, epq.EPQ_Q4_K, layers, head, dev, attn_ctx=CTX)
    got = []
    for i, t in enumerate(order):
        d.pos = CTX + i
        got.append(d.step(x[t:t + 1])[0].clone())
    torch.cuda.synchronize()
    return torch.stack(got), d.caches


def _tree(epq, dev, setup, ntok=NTOK):
    decode, layers, head, _ = setup
    caches = decode.kv_caches(CFG.layers, CFG.kv_heads, CFG.head_dim, CTX, CTX + 64, dev, seed=7)
    return decode.TreeDecoder(CFG, epq.EPQ_Q4_K, layers, head, decode.paged_cache(caches, CTX, page_size=32), ntok, dev)


def _near(a, b):
    # Every GEMV is within 1e-4 of the sum of its terms' magnitudes on either
    # side, about 1e-4 sqrt(512) < 2.3e-3 of a typical output; nine of them
    # follow one another, and a new row's Q8_0 code may fall to the other side
    # of a rounding (1 / 254 of its block's largest) where they differ.
    return (a - b).abs().max().item() <= 0.02 * b.abs().max().item()


def test_chain_equals_one_by_one(epq_lib, cuda_dev, setup, monkeypatch):
    want, _ = _one_by_one(epq_lib, cuda_dev, setup, range(NTOK), monkeypatch)
    t = _tree(epq_lib, cuda_dev, setup)
    parent = torch.arange(-1, NTOK - 1, dtype=torch.int32, device=cuda_dev).view(1, -1)
    got = t.forward(setup[3], parent)[0]
    assert t.status.item() == 0 and _near(got, want)


def test_tree_equals_its_paths(epq_lib, cuda_dev, setup, monkeypatch):
    tree = [-1, 0, 0, 1, 2, 4]
    t = _tree(epq_lib, cuda_dev, setup)
    got = t.forward(setup[3], torch.tensor([tree], dtype=torch.int32, device=cuda_dev))[0].clone()
    for path in ([0, 1, 3], [0, 2, 4, 5]):
        want, _ = _one_by_one(epq_lib, cuda_dev, setup, path, monkeypatch)
        assert _near(got[path], want)


def test_committed_step_and_graph(epq_lib, cuda_dev, setup, monkeypatch):
    """A greedy step along a tree that holds the model's own choices, twice:
    the second time captured in a graph."""
    tree = torch.tensor([[-1, 0, 0, 1, 2, 4]], dtype=torch.int32, device=cuda_dev)
    u = torch.zeros((1, NTOK), device=cuda_dev)
    t = _tree(epq_lib, cuda_dev, setup)
    best = t.forward(setup[3], tree)[0].argmax(1)
    tokens = torch.full((1, NTOK), -1, dtype=torch.int32, device=cuda_dev)
    tokens[0, 2], tokens[0, 4] = best[0], best[2]  # the path 0, 2, 4; token 5 is not the choice after 4
    path, n, nxt = t.step(setup[3], tokens, tree, u, temperature=0.0)
    assert path.tolist() == [[0, 2, 4, -1, -1, -1]] and n.item() == 3 and nxt.item() == best[4].item()
    assert t.cache.length.item() == CTX + 3
    _, caches = _one_by_one(epq_lib, cuda_dev, setup, [0, 2, 4], monkeypatch)
    D = CFG.head_dim
    for li in range(CFG.layers):
        for plane, want in enumerate((caches[li].k, caches[li].v)):
            rows = t.cache.pool[li, t.cache.table[0, :4].clamp(min=0).long(), :, plane].transpose(0, 1).reshape(CFG.kv_heads, -1, D + D // 16)
            assert torch.equal(rows[:, :CTX], want[:, :CTX])
            value = lambda r: (r[..., D // 16:].contiguous().view(torch.int8).float().view(CFG.kv_heads, 3, D // 32, 32)  # noqa: E731
                               * r[..., :D // 16].contiguous().view(torch.float16).float()[..., None])
            assert _near(value(rows[:, CTX:CTX + 3]), value(want[:, CTX:CTX + 3]))
    # the same step again, from the same state, as a graph
    t2 = _tree(epq_lib, cuda_dev, setup)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        t2.step(setup[3], tokens, tree, u, temperature=0.0)
    length = CTX
    for i in range(3):  # each replay commits its own path
        g.replay()
        torch.cuda.synchronize()
        length += t2.n_accept.item()
        assert t2.cache.length.item() == length and t2.status.item() == 0
        if i == 0:
            assert t2.path.tolist() == [[0, 2, 4, -1, -1, -1]] and torch.equal(t2.logits, t.logits)
    assert epq_lib.epq_device_error() == 0


def test_cache_without_room(epq_lib, cuda_dev, setup):
    """A step that cannot reserve its rows stores, accepts and commits nothing, on another stream too."""
    t = _tree(epq_lib, cuda_dev, setup)
    t.cache.refs[t.cache.refs == 0] = 1  # every other page is held elsewhere
    t.cache.length.fill_(95)             # one row is left in the last page
    pool = t.cache.pool.clone()
    parent = torch.arange(-1, NTOK - 1, dtype=torch.int32, device=cuda_dev).view(1, -1)
    tokens, u = torch.zeros((1, NTOK), dtype=torch.int32, device=cuda_dev), torch.zeros((1, NTOK), device=cuda_dev)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        path, n, nxt = t.step(setup[3], tokens, parent, u, temperature=0.0, stream=stream)
        torch.cuda.synchronize()
        assert t.status.item() == 1 and n.item() == 0 and nxt.item() == -1 and path.tolist() == [[-1] * NTOK]
        assert t.cache.length.item() == 95 and torch.equal(t.cache.pool, pool)
    assert epq_lib.epq_device_error() == 0


def test_step_on_the_default_stream_by_its_handle(epq_lib, cuda_dev, setup):
    """stream=0: every part of the step is queued on the default stream, after what is queued there."""
    t = _tree(epq_lib, cuda_dev, setup)
    parent = torch.arange(-1, NTOK - 1, dtype=torch.int32, device=cuda_dev).view(1, -1)
    tokens, u = torch.zeros((1, NTOK), dtype=torch.int32, device=cuda_dev), torch.zeros((1, NTOK), device=cuda_dev)
    want = [x.clone() for x in t.step(setup[3], tokens, parent, u, temperature=0.0)]
    length = t.cache.length.clone()
    t = _tree(epq_lib, cuda_dev, setup)
    t.status.fill_(1)  # what a part ahead of the reservation would take for its answer
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    got = t.step(setup[3], tokens, parent, u, temperature=0.0, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(t.cache.length, length)
    assert t.n_tok.item() == NTOK and epq_lib.epq_device_error() == 0
