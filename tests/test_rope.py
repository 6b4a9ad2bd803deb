"""Rotary positions and appended rows on the CPU: the frequencies against their
formulas, and the calls' refusals (argument errors are found on the host before
the device is looked at; tensors here live on the CPU and are never read)."""
import ctypes
import math

import pytest
import torch

EPQ_ERR_ARG, EPQ_ERR_SHAPE, EPQ_ERR_ALIGN = 1, 3, 4


@pytest.mark.parametrize("rot, base", [(2, 10000.0), (128, 10000.0), (64, 500000.0), (10, 1e6), (1024, 2.0)])
def test_frequencies(epq_lib, rot, base):
    f, m = epq_lib.epq_rope_frequencies(rot, base)
    assert f.dtype == torch.float64 and m == 1.0
    assert f.tolist() == pytest.approx([math.exp(-2 * j / rot * math.log(base)) for j in range(rot // 2)], rel=1e-13)


def test_scaled_frequencies(epq_lib):
    e, rot, base, ctx = epq_lib, 128, 10000.0, 4096.0
    f, _ = e.epq_rope_frequencies(rot, base)
    g, m = e.epq_rope_frequencies(rot, base, e.EPQ_ROPE_LINEAR, 4.0)
    assert m == 1.0 and torch.equal(g, f / 4.0)
    # by bands: pairs of more than 4 turns over the context stay, of less than 1 are stretched by the factor
    g, m = e.epq_rope_frequencies(rot, base, e.EPQ_ROPE_BANDS, 8.0, ctx)
    turns = ctx * f / (2 * math.pi)
    assert m == 1.0
    for j in range(rot // 2):
        t = float(turns[j])
        keep = min(max((t - 1) / 3, 0.0), 1.0)
        assert float(g[j]) == pytest.approx(float(f[j]) * (keep + (1 - keep) / 8), rel=1e-13)
    assert float(g[0]) == 1.0 and float(g[-1]) == float(f[-1]) / 8
    # by parts: a ramp in the pair's index, between the pairs of 32 turns and of 1
    g, m = e.epq_rope_frequencies(rot, base, e.EPQ_ROPE_PARTS, 8.0, ctx)
    assert m == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=1e-15)
    pair = lambda n: rot * math.log(ctx / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(pair(32.0)), math.ceil(pair(1.0))
    assert 0 < lo < hi < rot // 2
    for j in range(rot // 2):
        r = min(max((j - lo) / (hi - lo), 0.0), 1.0)
        assert float(g[j]) == pytest.approx(float(f[j]) * (r / 8 + 1 - r), rel=1e-13)
    # other borders
    g, _ = e.epq_rope_frequencies(rot, base, e.EPQ_ROPE_BANDS, 8.0, ctx, 2.0, 3.0)
    assert all(float(g[j]) == float(f[j]) for j in range(rot // 2) if turns[j] >= 3)
    assert all(float(g[j]) == float(f[j]) / 8 for j in range(rot // 2) if turns[j] <= 2)


@pytest.mark.parametrize("status, a", [
    (EPQ_ERR_SHAPE, (0, 1e4)), (EPQ_ERR_SHAPE, (3, 1e4)), (EPQ_ERR_SHAPE, (1026, 1e4)), (EPQ_ERR_ARG, (64, 1.0)),
    (EPQ_ERR_ARG, (64, math.nan)), (EPQ_ERR_ARG, (64, math.inf)), (EPQ_ERR_ARG, (64, 1e4, 4)),
    (EPQ_ERR_ARG, (64, 1e4, -1)), (EPQ_ERR_ARG, (64, 1e4, 1, 0.5)), (EPQ_ERR_ARG, (64, 1e4, 1, math.inf)),
    (EPQ_ERR_ARG, (64, 1e4, 2, 8.0, 0.0)), (EPQ_ERR_ARG, (64, 1e4, 2, 8.0, 4096.0, 32.0, 1.0)),
    (EPQ_ERR_ARG, (64, 1e4, 3, 8.0, 4096.0, 0.0, 4.0)),
])
def test_frequency_status(epq_lib, status, a):
    with pytest.raises(epq_lib.EpqError) as e:
        epq_lib.epq_rope_frequencies(*a)
    assert e.value.status == status


def _rope(epq, shape=(2, 3, 512), heads=4, rot=128, stream=0, n_pos=16, x=None, first=0, inter=False, **kw):
    t = epq.RopeTable.over(torch.zeros(n_pos, rot // 2, 2), first=first, interleaved=inter)
    return epq.epq_rope(torch.zeros(shape) if x is None else x, t, heads, stream=stream, **kw)


@pytest.mark.parametrize("status, kw", [
    (EPQ_ERR_SHAPE, dict(first=1)), (EPQ_ERR_SHAPE, dict(rot=130)), (EPQ_ERR_SHAPE, dict(rot=64, first=65)),
    (EPQ_ERR_SHAPE, dict(first=-1, rot=64)), (EPQ_ERR_SHAPE, dict(shape=(1, 2, 2048), heads=1)),
    (EPQ_ERR_SHAPE, dict(shape=(1, 65, 512), mask=torch.zeros(1, 65, dtype=torch.int64))),
    (EPQ_ERR_ARG, dict(shape=(1, 0, 512))), (EPQ_ERR_ARG, dict(shape=(0, 2, 512))),  # tensors of nothing have no address
])
def test_rope_status(epq_lib, status, kw):
    with pytest.raises(epq_lib.EpqError) as e:
        _rope(epq_lib, **kw)
    assert e.value.status == status


@pytest.mark.parametrize("kw", [
    dict(shape=(2, 1536)), dict(heads=5), dict(heads=0), dict(x=torch.zeros(2, 3, 512, dtype=torch.float64)),
    dict(x=torch.zeros(2, 3, 1024)[..., ::2]), dict(x=torch.zeros(1, 3, 512).expand(2, 3, 512)),
    dict(position=torch.zeros(2, 3)), dict(position=torch.zeros(2, 4, dtype=torch.int32)),
    dict(start=torch.zeros(3, dtype=torch.int32)), dict(start=torch.zeros(2, dtype=torch.int64)),
    dict(mask=torch.zeros(2, 3, dtype=torch.int32)), dict(n_tok=torch.zeros(2)),
    dict(out=torch.zeros(2, 3, 256)), dict(out=torch.zeros(2, 3, 512, dtype=torch.float16)),
])
def test_rope_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _rope(epq_lib, **kw)


def test_table_tensors(epq_lib):
    over = epq_lib.RopeTable.over
    for bad in (torch.zeros(4, 64), torch.zeros(4, 64, 3), torch.zeros(4, 64, 2, dtype=torch.float64),
                torch.zeros(4, 64, 4)[..., :2]):
        with pytest.raises(ValueError):
            over(bad)


def test_rope_c_status(epq_lib):
    """What the binding cannot pass."""
    lib, E = epq_lib.load(), epq_lib._lib
    t, x = torch.zeros(16, 64, 2), torch.zeros(2 * 3 * 512 + 4)
    r = E.Rotation(t.data_ptr(), 16, 128, 0, 0)
    o = E.RopeOpts()
    call = lambda r=r, x=x.data_ptr(), y=x.data_ptr(), n=(2, 3, 4, 128), o=o: lib.epq_rope(  # noqa: E731
        None if r is None else ctypes.byref(r), x, y, *n, ctypes.byref(o), None)
    assert call(r=None) == EPQ_ERR_ARG and call(x=None) == EPQ_ERR_ARG and call(y=None) == EPQ_ERR_ARG
    assert call(r=E.Rotation(None, 16, 128, 0, 0)) == EPQ_ERR_ARG
    assert call(r=E.Rotation(t.data_ptr(), 0, 128, 0, 0)) == EPQ_ERR_ARG
    assert call(r=E.Rotation(t.data_ptr(), 16, 127, 0, 0)) == EPQ_ERR_SHAPE
    assert call(r=E.Rotation(t.data_ptr() + 8, 16, 128, 0, 0)) == EPQ_ERR_ALIGN
    assert call(x=x.data_ptr() + 2) == EPQ_ERR_ALIGN
    assert call(n=(0, 3, 4, 128)) == EPQ_ERR_SHAPE and call(n=(2, 0, 4, 128)) == EPQ_ERR_SHAPE
    assert call(n=(2, 3, 65536, 128)) == EPQ_ERR_SHAPE and call(n=(1 << 16, 1 << 15, 4, 128)) == EPQ_ERR_SHAPE
    assert call(o=E.RopeOpts(y_ld=520)) == EPQ_ERR_ARG  # in place with other strides
    assert call(y=x.data_ptr() + 16, o=E.RopeOpts(y_ld=256)) == EPQ_ERR_ARG  # tokens of y overlap
    assert call(o=E.RopeOpts(x_ld=-512, y_ld=-512)) == EPQ_ERR_ARG
    f = torch.zeros(64, dtype=torch.float64)
    table = lambda f=f.data_ptr(), rot=128, m=1.0, n=16, t=t.data_ptr(): lib.epq_rope_table(f, rot, m, n, t, None)  # noqa: E731
    assert table(f=None) == EPQ_ERR_ARG and table(t=None) == EPQ_ERR_ARG and table(n=0) == EPQ_ERR_ARG
    assert table(m=math.nan) == EPQ_ERR_ARG and table(rot=7) == EPQ_ERR_SHAPE and table(n=1 << 31) == EPQ_ERR_SHAPE
    assert table(t=t.data_ptr() + 8) == EPQ_ERR_ALIGN


def _append(epq, ntok=3, layer=0, stream=0, n_seq=3, **kw):
    c = epq.PagedKVCache(2, 6, 2, 128, n_seq, 4, 16, "cpu")
    k = kw.pop("k", torch.zeros(n_seq, ntok, 256))
    v = kw.pop("v", torch.zeros(n_seq, ntok, 256))
    return epq.epq_pages_append(k, v, c, layer, stream=stream, **kw)


@pytest.mark.parametrize("status, kw", [
    (EPQ_ERR_ARG, dict(layer=2)), (EPQ_ERR_ARG, dict(layer=-1)), (EPQ_ERR_ARG, dict(ntok=0)),
    (EPQ_ERR_SHAPE, dict(ntok=65, mask=torch.zeros(3, 65, dtype=torch.int64))),
    (EPQ_ERR_ALIGN, dict(k=torch.zeros(3, 3, 258)[..., 2:], v=torch.zeros(3, 3, 258)[..., 2:])),
])
def test_append_status(epq_lib, status, kw):
    with pytest.raises(epq_lib.EpqError) as e:
        _append(epq_lib, **kw)
    assert e.value.status == status


def test_append_rotation_status(epq_lib):
    over = epq_lib.RopeTable.over
    for rope in (over(torch.zeros(4, 65, 2)), over(torch.zeros(4, 32, 2), first=96)):
        with pytest.raises(epq_lib.EpqError) as e:
            _append(epq_lib, rope=rope)
        assert e.value.status == EPQ_ERR_SHAPE


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(3, 768)), dict(k=torch.zeros(3, 3, 128)), dict(v=torch.zeros(3, 4, 256)),
    dict(k=torch.zeros(3, 3, 512)[..., :256]), dict(v=torch.zeros(3, 3, 256, dtype=torch.bfloat16)),
    dict(position=torch.zeros(3, 3, dtype=torch.int64)), dict(n_tok=torch.zeros(2, dtype=torch.int32)),
])
def test_append_tensors(epq_lib, kw):
    with pytest.raises(ValueError):
        _append(epq_lib, **kw)


def test_advance_tensors(epq_lib):
    c = epq_lib.PagedKVCache(2, 6, 2, 128, 3, 4, 16, "cpu")
    with pytest.raises(ValueError):
        epq_lib.epq_pages_advance(c, torch.zeros(2, dtype=torch.int32), stream=0)
    assert epq_lib.load().epq_pages_advance(ctypes.byref(c._p), None, None) == EPQ_ERR_ARG
