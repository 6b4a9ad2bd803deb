"""A prompt of several sequences some of which have no room: a sequence whose reservation was refused is left out with
n_tok 0, and what it shares with others stays as it is."""
import torch

import pytest

pytestmark = pytest.mark.gpu
KV, D, H, P, LAYERS = 2, 128, 4, 16, 2


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _step(epq, cache, qkv, n, rope):
    """A prompt's step as the documentation gives it."""
    status = epq.epq_pages_reserve(cache, n)
    n_tok = n * (status == 0)
    outs = []
    for layer in range(LAYERS):
        q, k, v = qkv[layer].split([H * D, KV * D, KV * D], dim=2)
        epq.epq_rope(q, rope, H, start=cache.length, n_tok=n_tok, out=q)
        epq.epq_pages_append(k, v, cache, layer, rope=rope, n_tok=n_tok)
        outs.append(epq.epq_attention_prompt(q, cache, layer, H, D ** -0.5, n_tok=n_tok))
    epq.epq_pages_advance(cache, n_tok)
    return status, outs


@pytest.mark.parametrize("spare", [0, 1])
def test_refused_sequence_leaves_its_siblings(epq_lib, spare):
    """Sequence 0 and its copy 1 share a last page that is partly filled; the pool has no page (or one, which is too few)
    for the copy's rows."""
    epq, rope = epq_lib, epq_lib.RopeTable(D, 256)
    g = torch.Generator(device="cuda").manual_seed(spare)
    new = lambda n: torch.randn(LAYERS, 3, n, (H + 2 * KV) * D, generator=g, device="cuda")  # noqa: E731
    cache = epq.PagedKVCache(LAYERS, 3 + spare, KV, D, 3, 8, P)
    status, _ = _step(epq, cache, new(40), _i32([40, 0, 0]), rope)
    assert status.tolist() == [0, 0, 0] and cache.length.tolist() == [40, 0, 0]
    epq.epq_pages_fork(cache, _i32([0]), _i32([1]))
    before = [t.clone() for t in (cache.pool, cache.table, cache.length, cache.refs)]
    extra = 30 if spare else 5  # 5 rows: the shared page's copy; 30: that and a page more
    status, outs = _step(epq, cache, new(30), _i32([0, extra, 0]), rope)
    assert status.tolist() == [0, 1, 0]
    for a, b in zip(before, (cache.pool, cache.table, cache.length, cache.refs)):
        assert torch.equal(a, b)
    assert not any(o.any() for o in outs)
    assert epq.epq_device_error() == 0
    # the sibling goes on once the copy is gone, and nothing of the refused rows is in its way
    epq.epq_pages_truncate(cache, _i32([-1, 0, -1]))
    status, _ = _step(epq, cache, new(8), _i32([8, 0, 0]), rope)
    assert status.tolist() == [0, 0, 0] and cache.length.tolist() == [48, 0, 0]
    page = cache.table[0, 2].item()
    assert torch.equal(cache.pool[:, page, :, :, :8], before[0][:, page, :, :, :8])
    assert epq.epq_device_error() == 0
