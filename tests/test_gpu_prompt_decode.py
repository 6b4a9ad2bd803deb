"""A sequence from its prompt to its constrained tokens (TreeDecoder): a prompt
at once against the same tokens decoded as chains of drafted ones, rotated
positions in a tree, and steps under penalties and a grammar, eager and captured.

Tolerances are those of the verification step's own test: every GEMV is within
1e-4 of the sum of its terms' magnitudes, about 2.3e-3 of a typical output; some
ten follow one another, and a row's Q8_0 code may fall to the other side of a
rounding (1 / 254 of its block's largest) where they differ."""
import dataclasses

import pytest
import torch

import synthetic
from synthetic.workloads import DenseDecode

pytestmark = pytest.mark.gpu

CFG = dataclasses.replace(DenseDecode(), layers=2, hidden=512, heads=4, kv_heads=2, inter=768, vocab=1024)


@pytest.fixture(scope="module")
def setup(epq_lib, cuda_dev):
    from moe_experts_gb300 import decode

    H, rows = CFG.hidden, CFG.q_rows + 2 * CFG.kv_rows
    pack = lambda r, c, seed: epq_lib.epq_quantize(epq_lib.EPQ_Q4_K, synthetic.student_t((r, c), seed=seed, scale=0.05).to(cuda_dev))  # noqa: E731
    layers = [(pack(rows, H, 10 * i), pack(H, CFG.q_rows, 10 * i + 1), pack(2 * CFG.inter, H, 10 * i + 2), pack(H, CFG.inter, 10 * i + 3))
              for i in range(CFG.layers)]
    head = pack(CFG.vocab, H, 99)
    emb = synthetic.normal((CFG.vocab, H), seed=5).to(cuda_dev)
    return decode, layers, head, emb


def _decoder(epq, dev, setup, ntok, rope=True, pages=24, max_pages=24):
    decode, layers, head, _ = setup
    cache = epq.PagedKVCache(CFG.layers, pages, CFG.kv_heads, CFG.head_dim, 1, max_pages, 16, dev)
    tab = epq.RopeTable(CFG.head_dim, 512, 10000.0, device=dev) if rope else None
    return decode.TreeDecoder(CFG, epq.EPQ_Q4_K, layers, head, cache, ntok, dev, rope=tab)


def _near(a, b):
    return (a - b).abs().max().item() <= 0.02 * b.abs().max().item()


def _chain(dev, n):
    return torch.arange(-1, n - 1, dtype=torch.int32, device=dev).view(1, -1)


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("n", [1, 8, 65, 100])
def test_prompt_equals_chains(epq_lib, cuda_dev, setup, n, rope):
    """All tokens at once, and eight at a time as drafted chains that are all accepted: the same cache up to roundings
    (layer 0, whose rows depend on the GEMVs alone: the same bytes), and the same logits."""
    ids = torch.randint(0, CFG.vocab, (n,), generator=torch.Generator().manual_seed(n))
    x = setup[3][ids.to(cuda_dev)]
    p = _decoder(epq_lib, cuda_dev, setup, 8, rope)
    got = p.prompt(x)
    assert p.status.item() == 0 and p.cache.length.item() == n and got.shape == (1, CFG.vocab)
    at = 0
    pool = table = None
    while at < n:
        m = min(8, n - at)
        t = _decoder(epq_lib, cuda_dev, setup, m, rope)
        if pool is not None:
            t.cache.pool.copy_(pool)
            t.cache.table.copy_(table)
            t.cache.refs.copy_(refs)
            t.cache.length.fill_(at)
        want = t.forward(x[at:at + m], _chain(cuda_dev, m))[0, -1:].clone()
        epq_lib.epq_pages_compact(t.cache, torch.arange(m, dtype=torch.int32, device=cuda_dev).view(1, -1),
                                  torch.tensor([m], dtype=torch.int32, device=cuda_dev))
        pool, table, refs = t.cache.pool.clone(), t.cache.table.clone(), t.cache.refs.clone()
        at += m
    assert _near(got, want)
    assert torch.equal(p.cache.table, table)
    rows = lambda pool, li: pool[li, table[0, : -(-n // 16)].long()].transpose(0, 2).reshape(2, CFG.kv_heads, -1, 136)[:, :, :n]  # noqa: E731
    assert torch.equal(rows(p.cache.pool, 0), rows(pool, 0))
    value = lambda r: r[..., 8:].contiguous().view(torch.int8).float() * r[..., :8].contiguous().view(torch.float16).float().repeat_interleave(32, -1)  # noqa: E731
    assert _near(value(rows(p.cache.pool, 1)), value(rows(pool, 1)))
    assert epq_lib.epq_device_error() == 0


def test_prompt_in_parts(epq_lib, cuda_dev, setup):
    x = setup[3][:90]
    a, b = _decoder(epq_lib, cuda_dev, setup, 4), _decoder(epq_lib, cuda_dev, setup, 4)
    want = a.prompt(x)
    b.prompt(x[:24])
    b.prompt(x[24:25])
    got = b.prompt(x[25:])
    assert _near(got, want) and b.cache.length.item() == 90


def test_tree_with_positions(epq_lib, cuda_dev, setup):
    """Behind a prompt, the logits of each path of a tree are those of the path alone as a chain."""
    tree = [-1, 0, 0, 1, 2, 4]
    x = setup[3][200:206]
    t = _decoder(epq_lib, cuda_dev, setup, 6)
    t.prompt(setup[3][:70])
    got = t.forward(x, torch.tensor([tree], dtype=torch.int32, device=cuda_dev))[0].clone()
    for path in ([0, 1, 3], [0, 2, 4, 5]):
        c = _decoder(epq_lib, cuda_dev, setup, len(path))
        c.prompt(setup[3][:70])
        assert _near(got[path], c.forward(x[path], _chain(cuda_dev, len(path)))[0])


def test_constrained_steps(epq_lib, cuda_dev, setup):
    """Greedy steps under a grammar and penalties, eager and as one captured graph: the same tokens; every one is allowed,
    and is the best of the adjusted logits, which the plain logits' would not all be."""
    dev = cuda_dev
    g = torch.Generator().manual_seed(4)
    words = torch.randint(-2**31, 2**31, (1, 4, CFG.vocab // 32), generator=g).int().to(dev)
    cons = dict(penalties=torch.tensor([[1.3, 0.5, 0.7]], device=dev), history=torch.arange(0, 60, dtype=torch.int32, device=dev).view(1, -1),
                history_len=torch.tensor([60], dtype=torch.int32, device=dev), prompt_len=torch.tensor([20], dtype=torch.int32, device=dev),
                bias_ids=torch.tensor([[3, 900]], dtype=torch.int32, device=dev), bias=torch.tensor([[-5.0, 2.0]], device=dev), allowed=words)
    tokens = torch.tensor([[7, 11, 13, 17]], dtype=torch.int32, device=dev)
    parent = torch.tensor([[-1, 0, 1, 0]], dtype=torch.int32, device=dev)
    u = torch.zeros((1, 4), device=dev)
    x = setup[3][tokens[0].long()]
    ts = [_decoder(epq_lib, dev, setup, 4) for _ in range(2)]
    for t in ts:
        t.prompt(setup[3][:60])
    ts[0].step(x, tokens, parent, u, temperature=0.0, constraints=cons)
    eager = [ts[0].path.clone(), ts[0].n_accept.clone(), ts[0].next_token.clone(), ts[0].logits.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ts[1].step(x, tokens, parent, u, temperature=0.0, constraints=cons)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, [ts[1].path, ts[1].n_accept, ts[1].next_token, ts[1].logits]):
        assert torch.equal(a, b)
    last = eager[0][0, int(eager[1]) - 1].item()
    assert int(eager[2]) == int(eager[3][0, last].argmax())
    assert int(words[0, last, int(eager[2]) // 32]) >> (int(eager[2]) % 32) & 1
    plain = _decoder(epq_lib, dev, setup, 4)
    plain.prompt(setup[3][:60])
    raw = plain.forward(x, parent)
    mask = epq_lib.epq_tree_mask(parent)
    assert torch.equal(epq_lib.epq_logits_adjust(raw, tokens=tokens, mask=mask, **cons), eager[3]) and not torch.equal(raw, eager[3])
    assert epq_lib.epq_device_error() == 0


def test_prompt_without_room(epq_lib, cuda_dev, setup):
    """A prompt that does not fit leaves the cache as it is, on another stream too."""
    t = _decoder(epq_lib, cuda_dev, setup, 4, pages=5)
    t.prompt(setup[3][:70])
    before = t.cache.pool.clone()
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        t.prompt(setup[3][:40], stream=stream)
        torch.cuda.synchronize()
        assert t.status.item() == 1 and t.cache.length.item() == 70 and torch.equal(t.cache.pool, before)
    t.prompt(setup[3][:10])
    assert t.status.item() == 0 and t.cache.length.item() == 80
    assert epq_lib.epq_device_error() == 0
