"""Refusals of the paged-cache and tree-verification calls.  Argument errors
are found on the host before the device is looked at, so these run without
one (tensors here live on the CPU and are never read)."""
import ctypes

import pytest
import torch

EPQ_ERR_ARG, EPQ_ERR_SHAPE, EPQ_ERR_ALIGN, EPQ_ERR_WORKSPACE = 1, 3, 4, 5


def _cache(epq, **kw):
    a = dict(n_layers=2, n_pages=6, n_kv_heads=2, head_dim=128, n_seq=3, max_pages=4, page_size=16, device="cpu")
    return epq.PagedKVCache(**{**a, **kw})


@pytest.mark.parametrize("bad", [dict(page_size=24), dict(page_size=8), dict(head_dim=96), dict(n_seq=257),
                                 dict(n_kv_heads=257)])
def test_cache_sizes(epq_lib, bad):
    with pytest.raises(ValueError):
        _cache(epq_lib, **bad)


def test_cache_over_wrong_tensors(epq_lib):
    c = _cache(epq_lib)
    with pytest.raises(ValueError):
        epq_lib.PagedKVCache.over(c.pool.view(torch.int8), c.table, c.length, c.refs)
    with pytest.raises(ValueError):
        epq_lib.PagedKVCache.over(c.pool, c.table.long(), c.length, c.refs)
    with pytest.raises(ValueError):
        epq_lib.PagedKVCache.over(c.pool, c.table, c.length[:2], c.refs)
    with pytest.raises(ValueError):
        epq_lib.PagedKVCache.over(c.pool[..., :100].contiguous(), c.table, c.length, c.refs)
    with pytest.raises(ValueError):
        epq_lib.PagedKVCache.over(c.pool[:, ::2], c.table, c.length, c.refs[:3])


def test_pages_status(epq_lib):
    lib, c = epq_lib.load(), _cache(epq_lib)
    p = ctypes.byref(c._p)
    n = c.length.data_ptr()
    assert lib.epq_pages_truncate(None, n, None) == EPQ_ERR_ARG
    assert lib.epq_pages_truncate(p, None, None) == EPQ_ERR_ARG
    assert lib.epq_pages_fork(p, n, None, 1, None, None) == EPQ_ERR_ARG
    assert lib.epq_pages_fork(p, n, n, 0, None, None) == EPQ_ERR_SHAPE
    assert lib.epq_pages_fork(p, n, n, 257, None, None) == EPQ_ERR_SHAPE
    assert lib.epq_pages_reserve(p, n, None, None) == EPQ_ERR_ARG
    assert lib.epq_pages_compact(p, n, n, 65, None) == EPQ_ERR_SHAPE
    assert lib.epq_pages_compact(p, n, None, 4, None) == EPQ_ERR_ARG
    q = type(c._p).from_buffer_copy(c._p)
    q.table += 4
    assert lib.epq_pages_truncate(ctypes.byref(q), n, None) == EPQ_ERR_ALIGN
    q = type(c._p).from_buffer_copy(c._p)
    q.work = None
    assert lib.epq_pages_truncate(ctypes.byref(q), n, None) == EPQ_ERR_ARG
    q = type(c._p).from_buffer_copy(c._p)
    q.max_pages = 1 << 27
    assert lib.epq_pages_truncate(ctypes.byref(q), n, None) == EPQ_ERR_SHAPE
    assert lib.epq_pages_work_bytes(ctypes.byref(q)) == 0


def test_pages_tensors(epq_lib):
    c = _cache(epq_lib)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        epq_lib.epq_pages_truncate(c, torch.zeros(2, dtype=torch.int32), stream=0)
    with pytest.raises(ValueError):
        epq_lib.epq_pages_reserve(c, torch.zeros(3), stream=0)
    with pytest.raises(ValueError):
        epq_lib.epq_pages_fork(c, i32[:1], i32[:2], stream=0)
    with pytest.raises(ValueError):
        epq_lib.epq_pages_compact(c, torch.zeros((2, 4), dtype=torch.int32), i32, stream=0)


def _attn(epq, c, ntok=4, heads=4, stream=0, layer=0, scale=0.1, **kw):
    D = c.head_dim
    q = kw.pop("q", torch.zeros(c.n_seq, ntok, heads * D))
    k = kw.pop("k", torch.zeros(c.n_seq, ntok, c.n_kv_heads * D))
    v = kw.pop("v", torch.zeros(c.n_seq, ntok, c.n_kv_heads * D))
    return epq.epq_attention_tree(q, k, v, c, layer, heads, scale, stream=stream, **kw)


@pytest.mark.parametrize("status, kw", [
    (EPQ_ERR_ARG, dict(layer=2)), (EPQ_ERR_ARG, dict(layer=-1)), (EPQ_ERR_ARG, dict(scale=0.0)),
    (EPQ_ERR_ARG, dict(scale=float("inf"))), (EPQ_ERR_ARG, dict(scale=float("nan"))),
    (EPQ_ERR_WORKSPACE, dict(workspace=torch.zeros(0, dtype=torch.uint8))),
    (EPQ_ERR_ALIGN, dict(q=torch.zeros(3, 4, 514)[..., 2:])),
    (EPQ_ERR_ALIGN, dict(q=torch.zeros(3 * 4 * 514)[1:1 + 4 * 3 * 512].view(3, 4, 512))),
])
def test_attention_status(epq_lib, status, kw):
    with pytest.raises(epq_lib.EpqError) as e:
        _attn(epq_lib, _cache(epq_lib), **kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(heads=3), dict(heads=34), dict(ntok=65), dict(ntok=0), dict(q=torch.zeros(3, 4, 512, dtype=torch.float64)),
    dict(q=torch.zeros(3, 4, 1024)[..., ::2]), dict(k=torch.zeros(3, 5, 256)), dict(k=torch.zeros(2, 4, 256)),
    dict(q=torch.zeros(1, 4, 512).expand(3, 4, 512)), dict(k=torch.zeros(3, 4, 512)[..., :256]),
    dict(mask=torch.zeros(3, 4, dtype=torch.int32)), dict(mask=torch.zeros(3, 5, dtype=torch.int64)),
    dict(n_tok=torch.zeros(4, dtype=torch.int32)), dict(out=torch.zeros(3, 4, 1024)[..., :512]),
])
def test_attention_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _attn(epq_lib, _cache(epq_lib), **kw)


def _verify(epq, nseq=2, ntok=3, vocab=40, stream=0, **kw):
    i32 = torch.zeros((nseq, ntok), dtype=torch.int32)
    a = dict(logits=torch.zeros(nseq, ntok, vocab), tokens=i32, parent=i32, u=torch.zeros(nseq, ntok))
    a.update(kw)
    return epq.epq_verify_tree(a.pop("logits"), a.pop("tokens"), a.pop("parent"), a.pop("u"), stream=stream, **a)


@pytest.mark.parametrize("status, kw", [
    (EPQ_ERR_ARG, dict(temperature=-1.0)), (EPQ_ERR_ARG, dict(temperature=float("nan"))),
    (EPQ_ERR_ARG, dict(temperature=float("inf"))), (EPQ_ERR_ARG, dict(u=None)),
    (EPQ_ERR_WORKSPACE, dict(workspace=torch.zeros(4, dtype=torch.uint8))),
    (EPQ_ERR_SHAPE, dict(ntok=65, workspace=torch.zeros(1 << 16, dtype=torch.uint8))),
])
def test_verify_status(epq_lib, status, kw):
    with pytest.raises(epq_lib.EpqError) as e:
        _verify(epq_lib, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(logits=torch.zeros(2, 3, 40, dtype=torch.float16)), dict(logits=torch.zeros(2, 3, 80)[..., ::2]),
    dict(tokens=torch.zeros(2, 3, dtype=torch.int64)), dict(u=torch.zeros(2, 4)), dict(draft=torch.zeros(2, 3, 41)),
    dict(n_tok=torch.zeros(3, dtype=torch.int32)), dict(path=torch.zeros(2, 2, dtype=torch.int32)), dict(vocab=262145),
    dict(ntok=65),
])
def test_verify_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _verify(epq_lib, **kw)


def test_tree_mask_refusals(epq_lib):
    lib = epq_lib.load()
    t = torch.zeros(8, dtype=torch.int64)
    assert lib.epq_tree_mask(None, 1, 1, t.data_ptr(), None) == EPQ_ERR_ARG
    assert lib.epq_tree_mask(t.data_ptr(), 1, 65, t.data_ptr(), None) == EPQ_ERR_SHAPE
    with pytest.raises(ValueError):
        epq_lib.epq_tree_mask(torch.zeros(1, 4, dtype=torch.int64), stream=0)


@pytest.mark.parametrize("call", [
    lambda epq, c, t: epq.epq_pages_truncate(c, t(3), stream=0),
    lambda epq, c, t: epq.epq_pages_fork(c, t(2), torch.zeros(2, dtype=torch.int32), stream=0),
    lambda epq, c, t: epq.epq_pages_fork(c, torch.zeros(2, dtype=torch.int32), t(2), stream=0),
    lambda epq, c, t: epq.epq_pages_fork(c, *[torch.zeros(2, dtype=torch.int32)] * 2, status=t(2), stream=0),
    lambda epq, c, t: epq.epq_pages_reserve(c, t(3), stream=0),
    lambda epq, c, t: epq.epq_pages_reserve(c, torch.zeros(3, dtype=torch.int32), t(3), stream=0),
    lambda epq, c, t: epq.epq_pages_compact(c, t(3, 4), torch.zeros(3, dtype=torch.int32), stream=0),
    lambda epq, c, t: epq.epq_pages_compact(c, torch.zeros((3, 4), dtype=torch.int32), t(3), stream=0),
    lambda epq, c, t: epq.epq_tree_mask(torch.zeros((3, 4), dtype=torch.int32), t(3, 4, dtype=torch.int64), stream=0),
    lambda epq, c, t: epq.PagedKVCache.over(c.pool, t(3, 4), c.length, c.refs),
    lambda epq, c, t: epq.PagedKVCache.over(c.pool, c.table, t(3), c.refs),
    lambda epq, c, t: epq.PagedKVCache.over(c.pool, c.table, c.length, t(6)),
    *[lambda epq, c, t, a=a: _attn(epq, c, layer=-1, **{a[0]: t(*a[1], dtype=a[2])}) for a in (
        ("q", (3, 4, 512), torch.float32), ("k", (3, 4, 256), torch.float32), ("v", (3, 4, 256), torch.float32),
        ("mask", (3, 4), torch.int64), ("n_tok", (3,), torch.int32), ("out", (3, 4, 512), torch.float32),
        ("workspace", (1 << 22,), torch.uint8))],
    *[lambda epq, c, t, a=a: _verify(epq, temperature=-1.0, **{a[0]: t(*a[1], dtype=a[2])}) for a in (
        ("logits", (2, 3, 40), torch.float32), ("draft", (2, 3, 40), torch.float32), ("tokens", (2, 3), torch.int32),
        ("parent", (2, 3), torch.int32), ("u", (2, 3), torch.float32), ("n_tok", (2,), torch.int32),
        ("path", (2, 3), torch.int32), ("n_accept", (2,), torch.int32), ("next_token", (2,), torch.int32),
        ("lse", (2, 3), torch.float32), ("workspace", (1 << 16,), torch.uint8))],
])
def test_tensors_of_another_device(epq_lib, call):
    """One tensor elsewhere than the others (on `meta`, next to a cache on the host) is refused before any launch."""
    with pytest.raises(ValueError):
        call(epq_lib, _cache(epq_lib), lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta"))


def test_workspace_of_one_byte_repeated(epq_lib):
    """A broadcast workspace has its size but not its memory."""
    with pytest.raises(ValueError):
        _attn(epq_lib, _cache(epq_lib), layer=-1, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24))
    with pytest.raises(ValueError):
        _verify(epq_lib, temperature=-1.0, workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 24))


def test_stream_arguments(epq_lib, monkeypatch):
    """Torch streams, objects with a handle, and handles; 0 is the default stream and no other."""
    from moe_experts_gb300 import _lib

    class Handle:
        cuda_stream = 4096

    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: ("external", h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    assert _lib._stream_object(0) == "default"
    assert _lib._stream_object(4096) == _lib._stream_object(Handle()) == ("external", 4096)


def test_verify_alignment(epq_lib):
    """Logits and draft rows may begin at any float, the workspace on 16 bytes (a bad address is never read)."""
    from moe_experts_gb300 import _lib

    lib, n = epq_lib.load(), 1 << 20
    call = lambda logits, draft, ws: lib.epq_verify_tree(  # noqa: E731
        logits, 40, n, n, n, 2, 3, ctypes.byref(_lib.VerifyOpts(draft, None, 1.0, 0, 0)), n, n, n, None, ws, 1 << 16, None)
    for at in ((n + 2, n, n), (n, n + 1, n), (n, n, n + 8)):
        assert call(*at) == EPQ_ERR_ALIGN
