"""GPU parity of the rotary positions and of appended rows.

epq_rope and epq_pages_append round each product and each sum to float32, so
against a table that is given both are compared bit for bit with the same
operations in torch; the table, and the rotation by it, also with the formula
in 64 bits: (c, s) are off by half a step of a value of at most the magnitude m
(2^-24 m) and an element by the table's error, two rounded products and a
rounded sum: (2^-24 + 2^-24 + 2^-24) m (|x0| + |x1|), with what is of second
order under another 2^-30 of it."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _pairs(rot, first, inter):
    j = torch.arange(rot // 2)
    return (first + 2 * j, first + 2 * j + 1) if inter else (first + j, first + rot // 2 + j)


def _turn32(x, table, pos, first, inter):
    """x [n_seq, ntok, heads, dim] float32, pos [n_seq, ntok]: each operation rounded."""
    one, two = _pairs(2 * table.shape[1], first, inter)
    t = table[pos.long()][:, :, None]
    y, a, b = x.clone(), x[..., one], x[..., two]
    y[..., one], y[..., two] = a * t[..., 0] - b * t[..., 1], b * t[..., 0] + a * t[..., 1]
    return y


@pytest.mark.parametrize("kind, rot, base, n_pos", [(0, 128, 10000.0, 5000), (1, 64, 10000.0, 40000), (2, 128, 500000.0, 131072), (3, 10, 1e6, 333),
                                                    (0, 2, 10000.0, 1)])
def test_table(epq_lib, kind, rot, base, n_pos):
    extra = dict(factor=8.0, context=8192.0) if kind else {}
    t = epq_lib.RopeTable(rot, n_pos, base, kind=kind, **extra)
    f, m = epq_lib.epq_rope_frequencies(rot, base, kind, **extra)
    a = torch.arange(n_pos, dtype=F64, device="cuda")[:, None] * f.cuda()
    want = torch.stack([a.cos(), a.sin()], 2) * m
    assert t.table.shape == want.shape
    assert ((t.table.double() - want).abs() <= 2.0 ** -24 * m * (1 + 2.0 ** -20)).all()


ROPES = [  # nseq, ntok, heads, dim, rot, first, interleaved
    (1, 1, 1, 2, 2, 0, False), (1, 1, 40, 128, 128, 0, False), (2, 3, 5, 128, 64, 64, True), (3, 13, 16, 256, 64, 0, False),
    (1, 517, 4, 80, 20, 60, False), (2, 5, 3, 80, 10, 7, True), (1, 2, 1, 1024, 1024, 0, False), (1, 2, 3, 1023, 6, 1000, True),
    (2, 70, 7, 96, 96, 0, True), (1, 9, 300, 64, 32, 32, False), (1, 4, 2, 128, 4, 124, False), (5, 1, 2, 33, 32, 1, False),
]


@pytest.mark.parametrize("case", ROPES)
def test_rope(epq_lib, case):
    nseq, ntok, heads, dim, rot, first, inter = case
    g = torch.Generator(device="cuda").manual_seed(sum(case[:6]))
    tab = epq_lib.RopeTable(rot, 3000, 10000.0, first=first, interleaved=inter)
    x = torch.randn(nseq, ntok, heads * dim, generator=g, device="cuda")
    start = torch.randint(0, 2000, (nseq,), generator=g, device="cuda").int()
    n_tok = torch.randint(0, ntok + 1, (nseq,), generator=g, device="cuda").int()
    pos = start[:, None] + torch.arange(ntok, device="cuda")
    x4 = x.view(nseq, ntok, heads, dim)
    want = _turn32(x4, tab.table, pos, first, inter).view_as(x)
    assert torch.equal(epq_lib.epq_rope(x, tab, heads, start=start), want)
    # positions that are given, in any order, and none
    perm = torch.randint(0, 3000, (nseq, ntok), generator=g, device="cuda").int()
    assert torch.equal(epq_lib.epq_rope(x, tab, heads, position=perm), _turn32(x4, tab.table, perm, first, inter).view_as(x))
    assert torch.equal(epq_lib.epq_rope(x, tab, heads), _turn32(x4, tab.table, (pos - start[:, None]), first, inter).view_as(x))
    # unused rows are copied, and left alone in place
    live = (torch.arange(ntok, device="cuda") < n_tok[:, None])[..., None]
    assert torch.equal(epq_lib.epq_rope(x, tab, heads, start=start, n_tok=n_tok), torch.where(live, want, x))
    y = x.clone()
    assert epq_lib.epq_rope(y, tab, heads, start=start, n_tok=n_tok, out=y) is y
    assert torch.equal(y, torch.where(live, want, x))
    # against the formula in 64 bits
    f, m = epq_lib.epq_rope_frequencies(rot, 10000.0)
    a = pos.double()[:, :, None, None] * f.cuda()
    one, two = _pairs(rot, first, inter)
    p, q = x4.double()[..., one], x4.double()[..., two]
    got = want.view(nseq, ntok, heads, dim).double()
    tol = 3 * 2.0 ** -24 * (p.abs() + q.abs()) * (1 + 2.0 ** -20)
    assert ((got[..., one] - (p * a.cos() - q * a.sin())).abs() <= tol).all()
    assert ((got[..., two] - (q * a.cos() + p * a.sin())).abs() <= tol).all()
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("off, ld", [(0, 0), (4, 4), (1, 3), (0, 2), (4, 1)])
def test_rope_views(epq_lib, off, ld):
    """Heads of a wider buffer, at any float, in place and into another; the rest stays."""
    g = torch.Generator(device="cuda").manual_seed(off + ld)
    tab = epq_lib.RopeTable(64, 100)
    W = off + 3 * 64 + ld
    buf = torch.randn(2, 6, W, generator=g, device="cuda")
    other = torch.full((6, 2, W + 4), 7.0, device="cuda")
    x = buf[..., off:off + 192]
    want = _turn32(x.reshape(2, 6, 3, 64), tab.table, torch.arange(6, device="cuda").expand(2, 6), 0, False).view(2, 6, 192)
    before = buf.clone()
    out = other.transpose(0, 1)[..., off:off + 192]  # sequences side by side in each token
    epq_lib.epq_rope(x, tab, 3, out=out)
    assert torch.equal(out, want) and torch.equal(buf, before)
    out.fill_(7.0)
    assert (other == 7.0).all()
    epq_lib.epq_rope(x, tab, 3, out=x)
    assert torch.equal(x, want)
    x.copy_(before[..., off:off + 192])
    assert torch.equal(buf, before)


def _tree(nseq, ntok, seed):
    r = np.random.default_rng(seed)
    parent = np.full((nseq, ntok), -1, dtype=np.int32)
    depth = np.zeros((nseq, ntok), dtype=np.int64)
    for s in range(nseq):
        for i in range(1, ntok):
            parent[s, i] = r.integers(max(0, i - 4), i)
            depth[s, i] = depth[s, parent[s, i]] + 1
    return parent, depth


@pytest.mark.parametrize("ntok", [1, 8, 64])
def test_rope_tree(epq_lib, ntok):
    parent, depth = _tree(2, ntok, ntok)
    mask = epq_lib.epq_tree_mask(torch.from_numpy(parent).cuda())
    tab = epq_lib.RopeTable(128, 300)
    x = torch.randn(2, ntok, 256, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    start = _i32([0, 200], "cuda")
    want = _turn32(x.view(2, ntok, 2, 128), tab.table, start[:, None] + torch.from_numpy(depth).cuda(), 0, False).view_as(x)
    assert torch.equal(epq_lib.epq_rope(x, tab, 2, start=start, mask=mask), want)


def test_rope_no_angle(epq_lib):
    """A position outside the table: NaN where it would have been turned, recorded, and nothing else changes."""
    tab = epq_lib.RopeTable(64, 10, first=32)
    x = torch.ones(1, 5, 2 * 128, device="cuda")
    pos = _i32([[9, 10, -1, 0, 2**31 - 1]], "cuda")
    y = epq_lib.epq_rope(x, tab, 2, position=pos).view(5, 2, 128)
    assert epq_lib.epq_device_error() == 6
    assert torch.equal(y[..., :32], x.view(5, 2, 128)[..., :32]) and torch.equal(y[..., 96:], x.view(5, 2, 128)[..., 96:])
    bad = torch.isnan(y[..., 32:96])
    assert bad[[1, 2, 4]].all() and not bad[[0, 3]].any()
    epq_lib.epq_rope(x, tab, 2, start=_i32([2**31 - 3], "cuda"))
    assert epq_lib.epq_device_error() == 6
    assert epq_lib.epq_device_error() == 0


def test_rope_graph_and_stream(epq_lib):
    """Captured and replayed on new inputs, and on a stream that is named."""
    tab = epq_lib.RopeTable(128, 4096)
    x, start = torch.randn(1, 8, 1280, device="cuda"), _i32([5], "cuda")
    out = torch.empty_like(x)
    st = torch.cuda.Stream()
    epq_lib.epq_rope(x, tab, 10, start=start, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        epq_lib.epq_rope(x, tab, 10, start=start, out=out)
    for k in range(3):
        x.normal_()
        start.fill_(1000 * k)
        graph.replay()
        want = epq_lib.epq_rope(x, tab, 10, start=start)
        st.wait_stream(torch.cuda.current_stream())
        other = epq_lib.epq_rope(x, tab, 10, start=start, stream=st)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(out, want) and torch.equal(out, other)


# ---------------------------------------------------------------- appended rows
def _rows(x):
    """float32 [..., D] -> the cache rows' bytes by the oracle's packer."""
    D = x.shape[-1]
    b = oracle.quantize(oracle.Q8_0, np.ascontiguousarray(x.reshape(-1, D), dtype=np.float32)).reshape(-1, D // 32, 34)
    return np.concatenate([b[:, :, :2].reshape(-1, D // 16), b[:, :, 2:].reshape(-1, D)], 1).reshape(*x.shape[:-1], D + D // 16)


def _cache(epq, layers, kv, D, P, lengths, ntok, seed):
    """A cache of random bytes with shuffled pages for lengths + ntok positions."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    each = [-(-(n + ntok) // P) for n in lengths]
    c = epq.PagedKVCache(layers, sum(each) + 2, kv, D, len(lengths), max(each) + 1, P)
    c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
    ids = torch.randperm(sum(each) + 2, generator=g, device="cuda").int()
    at = 0
    for s, n in enumerate(each):
        c.table[s, :n] = ids[at:at + n]
        at += n
    c.refs[ids[:at].long()] = 1
    c.length.copy_(_i32(lengths, "cuda"))
    return c


APPENDS = [  # kv, D, P, lengths, ntok, rot, first, interleaved
    (1, 128, 16, [0], 1, 128, 0, False), (8, 128, 64, [1037], 8, 128, 0, False), (2, 256, 32, [5, 64, 0], 70, 64, 192, True),
    (3, 128, 128, [127, 128], 130, 20, 3, False), (2, 128, 16, [15, 33], 17, 12, 1, True), (1, 256, 16, [300], 200, 256, 0, False),
    (16, 128, 16, [0, 333], 65, 64, 0, True), (2, 128, 64, [9], 5, 0, 0, False), (1, 256, 16, [3], 40, 34, 100, True),
]


@pytest.mark.parametrize("case", APPENDS)
def test_append(epq_lib, case):
    kv, D, P, lengths, ntok, rot, first, inter = case
    nseq = len(lengths)
    c = _cache(epq_lib, 2, kv, D, P, lengths, ntok, ntok)
    before = c.pool.clone()
    g = torch.Generator(device="cuda").manual_seed(kv + ntok)
    qkv = torch.randn(nseq, ntok, 3 * kv * D, generator=g, device="cuda")
    qkv[..., 5] = 0.0
    k, v = qkv[..., kv * D:2 * kv * D], qkv[..., 2 * kv * D:]
    n_tok = [ntok if s != 1 else ntok // 2 for s in range(nseq)]
    tab = epq_lib.RopeTable(rot, 1500, first=first, interleaved=inter) if rot else None
    epq_lib.epq_pages_append(k, v, c, 1, rope=tab, n_tok=_i32(n_tok, "cuda"))
    assert epq_lib.epq_device_error() == 0
    pos = c.length[:, None].long() + torch.arange(ntok, device="cuda")
    k4 = k.reshape(nseq, ntok, kv, D)
    if rot:
        k4 = _turn32(k4, tab.table, pos, first, inter)
    want = np.stack([_rows(k4.cpu().numpy()), _rows(v.reshape(nseq, ntok, kv, D).cpu().numpy())], 3)
    expect, table = before.cpu().numpy(), c.table.cpu().numpy()
    for s in range(nseq):
        for i in range(n_tok[s]):
            p = lengths[s] + i
            expect[1, table[s, p // P], :, :, p % P] = want[s, i]
    assert np.array_equal(c.pool.cpu().numpy(), expect)
    assert c.length.tolist() == lengths
    epq_lib.epq_pages_advance(c, _i32([n - 1 for n in n_tok], "cuda"))
    assert c.length.tolist() == [a + max(n - 1, 0) for a, n in zip(lengths, n_tok)]


def test_append_equals_rope_and_tree(epq_lib):
    """The rows that epq_attention_tree stores of keys turned by epq_rope are those of epq_pages_append, in a tree too."""
    parent, _ = _tree(2, 8, 3)
    mask = epq_lib.epq_tree_mask(torch.from_numpy(parent).cuda())
    a, b = (_cache(epq_lib, 1, 2, 128, 16, [37, 0], 8, 5) for _ in range(2))
    tab = epq_lib.RopeTable(128, 64)
    x = torch.randn(2, 8, 8 * 128, device="cuda")
    epq_lib.epq_pages_append(x[..., 512:768], x[..., 768:], a, 0, rope=tab, mask=mask)
    epq_lib.epq_rope(x[..., :768], tab, 6, start=b.length, mask=mask, out=x[..., :768])
    epq_lib.epq_attention_tree(x[..., :512], x[..., 512:768], x[..., 768:], b, 0, 4, 0.1, mask=mask)
    assert torch.equal(a.pool, b.pool)


def test_append_missing_pages_and_angles(epq_lib):
    """A row without a page is not stored; a key without an angle gets factors of NaN; both are recorded."""
    c = _cache(epq_lib, 1, 2, 128, 16, [10, 0], 20, 7)
    c.table[0, 1] = c.n_pages  # no such page: positions 16..31
    before = c.pool.clone()
    k = torch.randn(2, 20, 256, device="cuda")
    epq_lib.epq_pages_append(k, k, c, 0)
    assert epq_lib.epq_device_error() == 5
    changed = (c.pool != before).flatten(2).any(2)[0]
    assert set(changed.nonzero()[:, 0].tolist()) == {int(c.table[0, 0]), int(c.table[1, 0]), int(c.table[1, 1])}
    d = _cache(epq_lib, 1, 2, 128, 16, [0, 30], 2, 7)
    epq_lib.epq_pages_append(k[:, :2], k[:, :2], d, 0, rope=epq_lib.RopeTable(64, 31))
    assert epq_lib.epq_device_error() == 6
    f = d.pool[0, d.table[1, 1].item(), :, :, 15, :8].contiguous().view(torch.float16)  # position 31: [head, plane, 4]
    assert torch.isnan(f[:, 0]).all() and torch.isfinite(f[:, 1]).all()
    g = d.pool[0, d.table[1, 1].item(), :, :, 14, :8].contiguous().view(torch.float16)
    assert torch.isfinite(g).all()


def test_append_not_finite(epq_lib):
    """Infinities and NaN among the elements: the packer's bytes, in their own rows only."""
    c = _cache(epq_lib, 1, 1, 128, 16, [0], 6, 9)
    x = torch.randn(1, 6, 128, device="cuda")
    x[0, 1, 40], x[0, 2, 3], x[0, 3], x[0, 4, 77] = math.inf, math.nan, 0.0, 3.4e38
    epq_lib.epq_pages_append(x, x, c, 0)
    got = c.pool[0, c.table[0, 0].item(), 0].cpu().numpy()
    for i in (0, 5):
        w = _rows(x[0, i].cpu().numpy())
        assert np.array_equal(got[0, i], w) and np.array_equal(got[1, i], w)
    assert not got[0, 3].any()
    f = torch.from_numpy(got[0, :6, :8].copy()).view(torch.float16)
    assert torch.isinf(f[1, 1]) and torch.isinf(f[4, 2]) and torch.isfinite(f[[0, 2, 3, 5]]).all()


def test_advance_bounds(epq_lib):
    c = _cache(epq_lib, 1, 1, 128, 16, [0, 40, 3], 8, 11)
    epq_lib.epq_pages_advance(c, _i32([2**31 - 1, -5, 4], "cuda"))
    assert c.length.tolist() == [c.max_pages * 16, 40, 7]


def test_append_near_ties(epq_lib):
    """Elements at and next to the middle between two codes, over all mantissas of a factor and its exponents, subnormal
    halves too: the packer's bytes."""
    g = torch.Generator().manual_seed(3)
    n = 4096
    d = ((1024 + torch.randint(0, 1024, (n * 4,), generator=g)) * 2.0 ** torch.randint(-24, 5, (n * 4,), generator=g)).half()
    d[:256] = (torch.arange(1, 257) * 2.0 ** -24).half()
    x = (torch.randint(-127, 127, (n * 4, 32), generator=g) + 0.5).float() * d.float()[:, None]
    x = (x.view(torch.int32) + torch.randint(-3, 4, x.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    x[:, 0] = 127.0 * d.float()
    x[1::7, 0] *= 1.0 + 2.0 ** -12  # a factor that is rounded down: codes past 127
    x = x.view(1, n, 128)
    c = _cache(epq_lib, 1, 1, 128, 128, [0], n, 13)
    epq_lib.epq_pages_append(x.cuda(), x.flip(1).contiguous().cuda(), c, 0)
    rows = c.pool[0, c.table[0, : n // 128].long(), 0].transpose(0, 1).reshape(2, n, 136).cpu().numpy()
    assert np.array_equal(rows[0], _rows(x[0].numpy())) and np.array_equal(rows[1], _rows(x[0].flip(0).numpy()))


def test_host_tensors_are_refused(epq_lib):
    """Where there is a GPU, a call whose tensors are all on the host does not reach it."""
    with pytest.raises(ValueError):
        epq_lib.RopeTable(64, 10, device="cpu")
    t = epq_lib.RopeTable.over(torch.zeros(10, 32, 2))
    c = epq_lib.PagedKVCache(1, 4, 2, 128, 1, 2, 16, "cpu")
    k, n = torch.zeros(1, 3, 256), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: epq_lib.epq_rope(k, t, 2), lambda: epq_lib.epq_pages_append(k, k, c, 0), lambda: epq_lib.epq_pages_advance(c, n),
                 lambda: epq_lib.epq_attention_prompt(k, c, 0, 2, 0.1), lambda: epq_lib.epq_logits_adjust(k)):
        with pytest.raises(ValueError):
            call()


def test_append_two_at_once_and_none(epq_lib):
    """Two caches at the same time on two streams; a call in which no sequence has a row."""
    x = torch.randn(2, 600, 512, device="cuda")
    cs = [_cache(epq_lib, 1, 2, 128, 16, [5, 40], 600, 17) for _ in range(3)]
    tab = epq_lib.RopeTable(128, 1000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for c, st in zip(cs, streams):
        epq_lib.epq_pages_append(x[..., :256], x[..., 256:], c, 0, rope=tab, stream=st)
    torch.cuda.synchronize()
    before = cs[2].pool.clone()
    epq_lib.epq_pages_append(x[..., :256], x[..., 256:], cs[2], 0, rope=tab, n_tok=_i32([0, -4], "cuda"))
    assert torch.equal(cs[2].pool, before)
    epq_lib.epq_pages_append(x[..., :256], x[..., 256:], cs[2], 0, rope=tab, n_tok=_i32([600, 10000], "cuda"))
    assert torch.equal(cs[0].pool, cs[1].pool) and torch.equal(cs[0].pool, cs[2].pool)
    assert epq_lib.epq_device_error() == 0
