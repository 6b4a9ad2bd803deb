"""GPU parity of epq_attention_tree against the float64 oracle: the appended
rows bit for bit, the outputs within bounds that count float32 roundings
(oracle.tree.attention_bound)."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import tree as T

pytestmark = pytest.mark.gpu


def _rows(x):
    """float32 [..., D] -> cache rows [..., D + D/16]."""
    D = x.shape[-1]
    if x.size == 0:
        return np.zeros((*x.shape[:-1], D + D // 16), np.uint8)
    p = oracle.quantize(oracle.Q8_0, np.ascontiguousarray(x.reshape(-1, D), dtype=np.float32)).reshape(-1, D // 32, 34)
    r = np.concatenate([p[:, :, :2].reshape(len(p), -1), p[:, :, 2:].reshape(len(p), -1)], 1)
    return r.reshape(*x.shape[:-1], D + D // 16)


def _values(rows):
    D = rows.shape[-1] * 16 // 17
    if rows.size == 0:
        return np.zeros((*rows.shape[:-1], D), np.float32)
    d = np.ascontiguousarray(rows[..., :D // 16]).view("<f2").astype(np.float32)
    c = np.ascontiguousarray(rows[..., D // 16:]).view(np.int8).astype(np.float32)
    return (c.reshape(*d.shape, 32) * d[..., None]).reshape(*rows.shape[:-1], D)


class Case:
    def __init__(self, epq, dev, lengths, ntok, heads, kv, D, P, seed=0, layers=1, layer=0, spread=2.0, kscale=1.0, vscale=1.0,
                 max_extra=1, qscale=1.0):
        self.epq, self.dev, self.ntok, self.heads, self.kv, self.D, self.P, self.layer = epq, dev, ntok, heads, kv, D, P, layer
        rng = self.rng = np.random.default_rng(seed * 131 + sum(lengths) + ntok + D + P)
        nseq = len(lengths)
        each = [-(-(n + ntok) // P) for n in lengths]
        n_pages = sum(each) + 2
        self.c = epq.PagedKVCache(layers, n_pages, kv, D, nseq, max(each) + max_extra, P, dev)
        order, at = rng.permutation(n_pages), 0
        table = np.full((nseq, max(each) + max_extra), -1, np.int32)
        self.lengths, self.K, self.V = lengths, [], []
        pool = rng.integers(0, 256, tuple(self.c.pool.shape), dtype=np.uint8)
        # what no position holds: rows whose factors are NaN
        pool[..., :D // 16] = np.full(pool.shape[:-1] + (D // 32,), np.nan, np.float16).view(np.uint8)
        for s, n in enumerate(lengths):
            table[s, :each[s]] = order[at:at + each[s]]
            at += each[s]
            for c, scale in ((0, kscale), (1, vscale)):
                r = _rows((scale * rng.standard_normal((kv, n, D))).astype(np.float32)) if n else np.zeros((kv, 0, D + D // 16), np.uint8)
                (self.K, self.V)[c].append(r)
                for p in range(n):
                    pool[layer, table[s, p // P], :, c, p % P] = r[:, p]
        self.pool, self.table = pool, table
        self.c.pool.copy_(torch.from_numpy(pool))
        self.c.table.copy_(torch.from_numpy(table))
        self.c.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        w = (heads + 2 * kv) * D
        self.qkv = rng.standard_normal((nseq, ntok, w)).astype(np.float32)
        self.qkv[..., :heads * D] *= spread * qscale
        self.qkv[..., heads * D:(heads + kv) * D] *= kscale
        self.qkv[..., (heads + kv) * D:] *= vscale
        self.scale = 1.0 / (math.sqrt(D) * qscale * kscale)
        self.parents = [[-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, ntok)] for _ in range(nseq)]
        self.masks = [T.ancestors(p) for p in self.parents]

    def run(self, masks="tree", n_tok=None, ws=None, **kw):
        t = torch.from_numpy(self.qkv).to(self.dev)
        a, b = self.heads * self.D, (self.heads + self.kv) * self.D
        m = None
        if masks == "tree":
            m = self.masks
        elif masks is not None:
            m = masks
        mt = None if m is None else torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in m], dtype=torch.int64,
                                                 device=self.dev)
        nt = None if n_tok is None else torch.tensor(n_tok, dtype=torch.int32, device=self.dev)
        out = self.epq.epq_attention_tree(t[..., :a], t[..., a:b], t[..., b:], self.c, self.layer, self.heads, self.scale, mask=mt,
                                          n_tok=nt, workspace=ws, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, masks="tree", n_tok=None, ws=None, **kw):
        out = self.run(masks, n_tok, ws, **kw)
        got = out.cpu().numpy().reshape(len(self.lengths), self.ntok, self.heads, self.D).astype(np.float64)
        m = self.masks if masks == "tree" else masks or [[(2 << i) - 1 for i in range(self.ntok)]] * len(self.lengths)
        x = self.qkv.reshape(len(self.lengths), self.ntok, self.heads + 2 * self.kv, self.D)
        pool = self.pool.copy()
        G = self.heads // self.kv
        worst = 0.0
        for s, n in enumerate(self.lengths):
            live = self.ntok if n_tok is None else n_tok[s]
            assert np.array_equal(got[s, live:], np.zeros_like(got[s, live:]))
            new = [_rows(x[s, :live, self.heads + c * self.kv:self.heads + (c + 1) * self.kv]) for c in (0, 1)]  # [live, kv, row]
            for i in range(live):
                for c in (0, 1):
                    pool[self.layer, self.table[s, (n + i) // self.P], :, c, (n + i) % self.P] = new[c][i]
            for h in range(self.kv):
                K, V = (np.concatenate([_values((self.K, self.V)[c][s][h]), _values(new[c][:, h])]) for c in (0, 1))
                for g in range(h * G, (h + 1) * G):
                    ref, wabs, smag = T.tree_attention_f64(x[s, :live, g], K, V, n, m[s], self.scale)
                    e = np.abs(got[s, :live, g] - ref)
                    b = T.attention_bound(wabs, smag, n + live, self.D)
                    assert (e <= b).all(), f"seq {s} head {g}: {(e / b).max():.3g} at {np.unravel_index((e / b).argmax(), e.shape)}"
                    worst = max(worst, float((e / b).max()) if e.size else 0.0)
        assert np.array_equal(self.c.pool.cpu().numpy(), pool), "the cache holds other rows"
        assert self.epq.epq_device_error() == 0
        assert torch.equal(out, self.run(masks, n_tok, ws, **kw)), "not reproducible"
        return out


SHAPES = [
    # lengths, ntok, heads, kv, D, page
    ([37], 1, 32, 8, 128, 64),
    ([0], 1, 4, 2, 128, 16),
    ([0], 64, 8, 2, 128, 64),
    ([1], 2, 2, 2, 256, 32),
    ([63, 64, 65], 8, 8, 2, 128, 64),
    ([127, 128, 129, 0], 5, 4, 4, 128, 128),
    ([300, 17], 13, 6, 2, 128, 16),
    ([1024], 8, 32, 8, 128, 64),
    ([1999], 64, 16, 4, 128, 32),
    ([513, 31], 33, 16, 1, 256, 64),
    ([777], 7, 15, 3, 256, 16),
    ([4000], 16, 8, 8, 128, 64),
    ([3, 0, 1, 2, 5, 100], 3, 7, 1, 128, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)).replace(" ", ""))
def test_parity(epq_lib, cuda_dev, shape):
    Case(epq_lib, cuda_dev, *shape).check()


@pytest.mark.parametrize("group", range(1, 17))
def test_groups_and_row_counts(epq_lib, cuda_dev, group):
    """Every group size; token counts on both sides of the row tiles."""
    for ntok in (1, 3, 16 // group + 1, 64 if group % 5 == 0 else 17):
        Case(epq_lib, cuda_dev, [70], ntok, group, 1, 128, 32, seed=group).check()


def test_chain_and_ragged(epq_lib, cuda_dev):
    c = Case(epq_lib, cuda_dev, [33, 500, 0], 9, 8, 4, 128, 16)
    c.check(masks=None)
    Case(epq_lib, cuda_dev, [33, 500, 0], 9, 8, 4, 128, 16).check(masks=None, n_tok=[9, 0, 4])
    Case(epq_lib, cuda_dev, [33, 500, 0], 9, 8, 4, 128, 16).check(n_tok=[1, 9, 0])


def test_masks_that_leave_nothing(epq_lib, cuda_dev):
    """An empty mask: the cached positions alone, or 0 without any; bits past the tree say nothing."""
    c = Case(epq_lib, cuda_dev, [0, 20], 6, 4, 2, 128, 16)
    m = [[0, 2, 1 << 5, (1 << 64) - 1 - 63, 0, 8], [0, 0, 0, (1 << 64) - 1, 2, 1 << 63]]
    out = c.check(masks=m)
    assert not out[0, 0].any() and not out[0, 3].any() and not out[0, 4].any() and out[1, 0].any()


def test_not_finite_where_masked(epq_lib, cuda_dev):
    """Drafted keys and values that are NaN or infinite stay with the tokens that attend to them."""
    c = Case(epq_lib, cuda_dev, [100], 6, 8, 2, 128, 16)
    a = c.heads * c.D
    clean = c.run(masks=[[1, 3, 4, 12, 17, 33]])
    c.qkv[0, 2, a:a + 40] = np.nan
    c.qkv[0, 2, a + 256:] = np.inf
    c.qkv[0, 3, a:] = -np.inf
    got = c.run(masks=[[1, 3, 4, 12, 17, 33]])
    for i in (0, 1, 4, 5):
        assert torch.equal(got[0, i], clean[0, i])
    assert not torch.isfinite(got[0, 2]).all() and not torch.isfinite(got[0, 3]).all()
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("what", ["key", "value"])
def test_rows_of_nan(epq_lib, cuda_dev, what):
    """A drafted key or value of nothing but NaN: NaN for the tokens that attend to it, no other bit changed."""
    c = Case(epq_lib, cuda_dev, [70], 6, 8, 2, 128, 16)
    masks = [[1, 3, 4, 12, 17, 33]]
    clean = c.run(masks=masks)
    a = c.heads * c.D + (c.kv * c.D if what == "value" else 0)
    c.qkv[0, 2, a:a + c.kv * c.D] = np.nan
    got = c.run(masks=masks)
    for i in (0, 1, 4, 5):
        assert torch.equal(got[0, i], clean[0, i])
    assert torch.isnan(got[0, 2]).all() and torch.isnan(got[0, 3]).all()
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("kw", [dict(vscale=1e-4), dict(vscale=3e4), dict(kscale=1e-3), dict(kscale=1e3), dict(qscale=1e-12),
                                dict(qscale=1e12), dict(spread=40.0)], ids=str)
def test_magnitudes(epq_lib, cuda_dev, kw):
    """Small and large keys, values and queries, and scores that leave one position all the weight."""
    Case(epq_lib, cuda_dev, [290], 5, 8, 2, 128, 32, **kw).check()


def test_uneven_values(epq_lib, cuda_dev):
    """Value rows of very different size: zero rows, and one that carries the result with a small weight."""
    c = Case(epq_lib, cuda_dev, [200], 4, 4, 1, 128, 16)
    for p in range(200):
        f = 0.0 if p % 7 == 0 else 10.0 ** (p % 5 - 2)
        r = _rows(f * c.rng.standard_normal((1, 128)).astype(np.float32))
        c.V[0][:, p] = r
        c.pool[0, c.table[0, p // 16], :, 1, p % 16] = r
    c.c.pool.copy_(torch.from_numpy(c.pool))
    c.check()


def test_layers_and_kept_workspace(epq_lib, cuda_dev):
    """Another layer of a deeper cache; one workspace for calls of different lengths."""
    c = Case(epq_lib, cuda_dev, [129, 40], 8, 8, 2, 128, 32, layers=3, layer=2)
    ws = epq_lib.epq_attention_tree_workspace(c.c, 8, 8)
    c.check(ws=ws)
    for n in ([128, 3], [0, 0], [5, 40]):
        c.c.length.copy_(torch.tensor(n, dtype=torch.int32))
        short = c.run(ws=ws)
        assert torch.equal(short, c.run())


def test_other_stream_and_graph(epq_lib, cuda_dev):
    c = Case(epq_lib, cuda_dev, [600], 8, 16, 4, 128, 64)
    want = c.check()
    t = torch.from_numpy(c.qkv).to(cuda_dev)
    a, b = c.heads * c.D, (c.heads + c.kv) * c.D
    ws = epq_lib.epq_attention_tree_workspace(c.c, c.heads, c.ntok)
    parent = torch.tensor(c.parents, dtype=torch.int32, device=cuda_dev)
    out, mask = torch.zeros_like(want), torch.zeros((1, 8), dtype=torch.int64, device=cuda_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        epq_lib.epq_tree_mask(parent, mask)
        epq_lib.epq_attention_tree(t[..., :a], t[..., a:b], t[..., b:], c.c, 0, c.heads, c.scale, mask=mask, out=out, workspace=ws)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_missing_pages(epq_lib, cuda_dev):
    """Positions without a page are left out and recorded; a bad id is not followed."""
    c = Case(epq_lib, cuda_dev, [40], 4, 4, 2, 128, 16, max_extra=0)
    for bad in (-1, 1 << 20):
        c.c.table[0, 1] = bad
        got = c.run()
        assert torch.isfinite(got).all() and epq_lib.epq_device_error() == 5
    before = c.c.pool.clone()
    c.c.table[0, 2] = -1  # the page of the new rows
    got = c.run()
    assert torch.isfinite(got).all() and epq_lib.epq_device_error() == 5
    assert torch.equal(before, c.c.pool)
    c.c.length.fill_(1 << 30)  # held to the table: the new rows have no place
    got = c.run()
    assert torch.isfinite(got).all() and epq_lib.epq_device_error() == 5
    assert torch.equal(before, c.c.pool)


def test_pages_past_32_bits(epq_lib, cuda_dev):
    """Pages more than 2^32 bytes into a pool, of its second layer: the same outputs, stored and committed rows."""
    c = Case(epq_lib, cuda_dev, [300], 8, 16, 8, 128, 128)
    want = c.check()
    ids = torch.tensor([16999, 15800, 16001], device=cuda_dev)
    big = epq_lib.PagedKVCache(2, 17000, 8, 128, 1, c.c.max_pages, 128, cuda_dev)
    small = c.c.table[0, :3].long()
    big.table[0, :3] = ids.int()
    big.pool[1, ids] = c.c.pool[0, small]
    big.length.fill_(300)
    big.refs[ids] = 1
    big.pool[1, ids[2], :, :, 44:52] = 0  # the new rows
    c.c, kept, c.layer = big, c.c, 1
    assert torch.equal(c.run(), want) and torch.equal(big.pool[1, ids], kept.pool[0, small])
    path = torch.tensor([[0, 2, 3, 6, 7, -1, -1, -1]], dtype=torch.int32, device=cuda_dev)
    n = torch.tensor([5], dtype=torch.int32, device=cuda_dev)
    for cache in (kept, big):
        epq_lib.epq_pages_compact(cache, path, n)
        assert cache.length.tolist() == [305]
    assert torch.equal(big.pool[1, ids], kept.pool[0, small]) and epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("largest", [6, 14])
@pytest.mark.parametrize("apart", [10, 14, 18, 22])
def test_uneven_blocks(epq_lib, cuda_dev, apart, largest, D):
    """Blocks of one value row that are powers of two apart, the largest factor below and above 2: the same blocks in
    every row, then others from row to row.  The outputs of the small blocks count by themselves."""
    for moving in (False, True):
        c = Case(epq_lib, cuda_dev, [300], 5, 4, 1, D, 32, seed=apart)
        NB, a = D // 32, (c.heads + c.kv) * D
        up = 2.0 ** largest

        def scaled(x, p):
            f = np.array([up if (b + (p if moving else 0)) % 3 == 0 else up * 2.0 ** (-apart / (1 + b % 2)) for b in range(NB)])
            return (x.reshape(-1, NB, 32) * f[:, None]).reshape(x.shape).astype(np.float32)

        for p in range(300):
            r = _rows(scaled(c.rng.standard_normal((1, D)), p))
            c.V[0][:, p] = r
            c.pool[0, c.table[0, p // 32], :, 1, p % 32] = r
        for i in range(c.ntok):
            c.qkv[0, i, a:] = scaled(c.qkv[0, i, a:], 300 + i)
        c.c.pool.copy_(torch.from_numpy(c.pool))
        c.check()


def _check_without(epq, c, gone):
    """The outputs are those of a cache without the positions of sequence s in its pages gone[s]."""
    for s, pages in enumerate(gone):
        c.c.table[s, pages] = -1
    got = c.run().cpu().numpy().reshape(len(c.lengths), c.ntok, c.heads, c.D).astype(np.float64)
    assert epq.epq_device_error() == (5 if any(gone) else 0)
    x = c.qkv.reshape(len(c.lengths), c.ntok, c.heads + 2 * c.kv, c.D)
    for s, n in enumerate(c.lengths):
        keep = [p for p in range(n) if p // c.P not in gone[s]]
        for g in range(c.heads):
            h = g // (c.heads // c.kv)
            K, V = (np.concatenate([_values((c.K, c.V)[k][s][h][keep]), _values(_rows(x[s, :, c.heads + k * c.kv + h]))])
                    for k in (0, 1))
            ref, wabs, smag = T.tree_attention_f64(x[s, :, g], K, V, len(keep), c.masks[s], c.scale)
            e, b = np.abs(got[s, :, g] - ref), T.attention_bound(wabs, smag, len(keep) + c.ntok, c.D)
            assert (e <= b).all(), f"seq {s} head {g}: {(e / b).max():.3g}"


@pytest.mark.parametrize("low", [0.0, 10.0, 300.0])
@pytest.mark.parametrize("P", [16, 64, 128])
def test_missing_pages_leave_the_others(epq_lib, cuda_dev, P, low):
    """Missing pages in sequences of many tiles, several to a CTA, the first ones among them; scores near 0 and far below
    it.  A sequence whose every page is missing attends to its drafted tokens alone."""
    lengths, heads, kv, D = [2500, 2437, 700, 2000], 16, 16, 128
    c = Case(epq_lib, cuda_dev, lengths, 2, heads, kv, D, P, max_extra=0)
    if low:  # every score is about -low: keys near one direction, queries against it
        axis = c.rng.choice([-1.0, 1.0], D)
        c.qkv[..., :heads * D] = np.tile(-low * axis, heads) * (1 + 0.02 * c.rng.standard_normal(c.qkv[..., :heads * D].shape))
        c.scale = 1.0 / D
        c.qkv[..., heads * D:(heads + kv) * D] = np.tile(axis, kv) * (1 + 0.02 * c.rng.standard_normal(
            c.qkv[..., heads * D:(heads + kv) * D].shape))
        for s, n in enumerate(lengths):
            r = _rows((axis * (1 + 0.02 * c.rng.standard_normal((kv, n, D)))).astype(np.float32))
            c.K[s] = r
            for p in range(n):
                c.pool[0, c.table[s, p // P], :, 0, p % P] = r[:, p]
        c.c.pool.copy_(torch.from_numpy(c.pool))
    last = [n // P for n in lengths]
    gone = [[j for j in range(last[0]) if j * P // 128 % 3 == 0],         # every third stretch of 128 positions
            list(range(last[1] - 3)),                                     # all but the last ones
            list(range(last[2])) + ([last[2]] if 700 % P else []), []]  # all
    _check_without(epq_lib, c, gone)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("n", [1, 5, 300])
def test_small_weight_on_a_small_value(epq_lib, cuda_dev, n, D):
    """One position has nearly all the weight and the largest value, but zeros among its elements: those elements are
    made by the others' small weights on rows that are 2^5 to 2^10 smaller, and count by themselves."""
    for ratio in (5, 8, 10):
        c = Case(epq_lib, cuda_dev, [n], 4, 4, 1, D, 32, seed=ratio, spread=6.0)
        a, k = (c.heads + c.kv) * D, c.heads * D
        axis = c.rng.choice([-1.0, 1.0], D)
        # the last committed position takes the weight: 2^-11 and less for the others
        keys = 0.3 * c.rng.standard_normal((1, n, D))
        keys[0, n - 1] = axis
        c.K[0] = _rows(keys.astype(np.float32))
        c.qkv[0, :, k:a] = 0.3 * c.rng.standard_normal((c.ntok, D))
        c.qkv[0, :, :k] = np.tile(axis * 8.0 / math.sqrt(D), c.heads) + c.rng.standard_normal((c.ntok, k)) * 0.5
        v = 2.0 ** -ratio * c.rng.standard_normal((1, n, D))
        v[0, n - 1] = np.where(np.arange(D) % 3 == 0, 0.0, c.rng.standard_normal(D))
        c.V[0] = _rows(v.astype(np.float32))
        c.qkv[0, :, a:] = 2.0 ** -ratio * c.rng.standard_normal((c.ntok, D))
        for p in range(n):
            c.pool[0, c.table[0, p // 32], :, 0, p % 32] = c.K[0][:, p]
            c.pool[0, c.table[0, p // 32], :, 1, p % 32] = c.V[0][:, p]
        c.c.pool.copy_(torch.from_numpy(c.pool))
        c.check()
