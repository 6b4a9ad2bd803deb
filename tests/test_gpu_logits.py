"""GPU parity of epq_logits_adjust: bit for bit with the same float32 operations
in numpy, token by token from lists; and with the formula in 64 bits, where each
of the five operations is off by at most half a step, 2^-24 of its result."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F = np.float32
U = 2.0 ** -24


def _reference(x, pen=None, hist=None, hlen=None, plen=None, tokens=None, mask=None, n_tok=None, ids=None, bias=None, allowed=None):
    """(float32 result, float64 result, its tolerance)"""
    nseq, ntok, vocab = x.shape
    y, z, tol = x.copy(), x.astype(np.float64), np.zeros(x.shape)
    for s in range(nseq):
        live = ntok if n_tok is None else min(max(int(n_tok[s]), 0), ntok)
        r, f, p = (F(1), F(0), F(0)) if pen is None else pen[s]
        n = 0 if hist is None else hist.shape[1] if hlen is None else min(max(int(hlen[s]), 0), hist.shape[1])
        given = 0 if plen is None else min(max(int(plen[s]), 0), n)
        add = {}
        for v, b in zip([] if ids is None else ids[s].tolist(), [] if bias is None else bias[s]):
            if 0 <= v < vocab:
                add[v] = b
        for i in range(live):
            count, read = {}, set()
            for k in range(n):
                v = int(hist[s, k])
                if k < given:
                    read.add(v)
                else:
                    count[v] = count.get(v, 0) + 1
            for j in range(live if tokens is not None else 0):
                if (j <= i) if mask is None else int(mask[s, i]) >> j & 1:
                    v = int(tokens[s, j])
                    count[v] = count.get(v, 0) + 1
            for v in set(add) | set(count) | read:
                if not 0 <= v < vocab:
                    continue
                l, d = y[s, i, v], z[s, i, v]
                t = 0.0
                with np.errstate(all="ignore"):
                    if v in add:
                        l, d = F(l + add[v]), d + float(add[v])
                        t += U * abs(d)
                    if v in count or v in read:
                        l = F(l / r) if l > 0 else F(l * r)
                        grow = 1 / float(r) if d > 0 else float(r)
                        t = t * max(grow, 1 / float(r), float(r)) + U * abs(d * grow)
                        d = d * grow
                    if v in count:
                        c = F(count[v])
                        l = F(l - F(F(f * c) + p))
                        t += U * (abs(float(f) * count[v]) + abs(float(f) * count[v] + float(p)))
                        d = d - (float(f) * count[v] + float(p))
                        t += U * abs(d)
                y[s, i, v], z[s, i, v], tol[s, i, v] = l, d, t * (1 + 2.0 ** -10)
            if allowed is not None:
                bits = (allowed[s, i].astype(np.int64)[np.arange(vocab) // 32] >> (np.arange(vocab) % 32)) & 1
                y[s, i, bits == 0] = z[s, i, bits == 0] = -math.inf
    return y, z, tol


def _same(got, want):
    y, z, tol = want
    assert np.array_equal(got, y, equal_nan=True)
    fine = np.isfinite(z)
    assert np.array_equal(np.isneginf(got), np.isneginf(z))
    assert (np.abs(got.astype(np.float64) - z)[fine] <= tol[fine]).all()


def _gpu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _run(epq, x, pen=None, hist=None, hlen=None, plen=None, tokens=None, mask=None, n_tok=None, ids=None, bias=None, allowed=None, out=None):
    return epq.epq_logits_adjust(_gpu(x), _gpu(pen), _gpu(hist), _gpu(hlen), _gpu(plen), _gpu(tokens), _gpu(mask), _gpu(n_tok), _gpu(ids),
                                 _gpu(bias), _gpu(allowed), out).cpu().numpy()


def _inputs(nseq, ntok, vocab, H, B, seed, tree=True, grammar=True):
    r = np.random.default_rng(seed)
    i32 = np.int32
    a = dict(x=(3 * r.standard_normal((nseq, ntok, vocab))).astype(F))
    a["pen"] = np.stack([1 + 0.5 * r.random(nseq) - 0.2, r.random(nseq) - 0.3, r.random(nseq) - 0.3], 1).astype(F)
    if H:
        a["hist"] = (vocab * r.random((nseq, H)) ** 4).astype(i32)
        a["hist"][:, ::7] = r.integers(-5, vocab + 5, a["hist"][:, ::7].shape)
        a["hlen"] = r.integers(-1, H + 2, nseq).astype(i32)
        a["plen"] = r.integers(-1, H + 2, nseq).astype(i32)
    a["tokens"] = r.integers(0, max(1, min(vocab, 6)), (nseq, ntok)).astype(i32)
    a["tokens"][:, 1::5] = r.integers(-3, vocab + 3, a["tokens"][:, 1::5].shape)
    if tree:
        m = np.zeros((nseq, ntok), dtype=np.int64)
        for s in range(nseq):
            for i in range(ntok):
                m[s, i] = (m[s, r.integers(0, i)] if i else 0) | np.int64(np.uint64(1 << i).astype(np.int64))
        a["mask"] = m
    a["n_tok"] = r.integers(0, ntok + 2, nseq).astype(i32)
    a["n_tok"][0] = ntok
    if B:
        a["ids"] = r.integers(-2, vocab + 2, (nseq, B)).astype(i32)
        a["ids"][:, -1] = a["ids"][:, 0]  # named twice: the last counts
        a["bias"] = (4 * r.standard_normal((nseq, B))).astype(F)
    if grammar:
        a["allowed"] = r.integers(-2**31, 2**31, (nseq, ntok, -(-vocab // 32))).astype(i32)
        a["allowed"][:, :, ::3] = 0
    return a


CASES = [(1, 1, 1, 0, 0), (1, 1, 1, 3, 2), (1, 1, 33, 5, 1), (2, 3, 4095, 40, 7), (1, 8, 4096, 300, 9), (3, 13, 4097, 100, 300), (2, 64, 9001, 1000, 20),
         (1, 1, 50001, 1037, 8), (4, 5, 12290, 17, 0), (1, 1, 128256, 0, 5), (5, 2, 31, 64, 40)]


@pytest.mark.parametrize("case", CASES)
def test_adjust(epq_lib, case):
    a = _inputs(*case, seed=sum(case))
    _same(_run(epq_lib, **a), _reference(**a))


@pytest.mark.parametrize("leave", ["pen", "hist", "hlen", "plen", "tokens", "mask", "n_tok", "ids", "allowed", "all"])
def test_parts(epq_lib, leave):
    """Without one of the options, and with none."""
    a = _inputs(2, 9, 5000, 50, 6, seed=3)
    drop = {"hist": ["hist", "hlen", "plen"], "ids": ["ids", "bias"], "all": [k for k in a if k != "x"]}.get(leave, [leave])
    a = {k: v for k, v in a.items() if k not in drop}
    _same(_run(epq_lib, **a), _reference(**a))


def test_in_place_and_unused_rows(epq_lib):
    a = _inputs(3, 7, 4500, 20, 3, seed=5)
    a["n_tok"][:] = [7, 0, 3]
    x = _gpu(a["x"])
    args = [_gpu(a[k]) for k in ("pen", "hist", "hlen", "plen", "tokens", "mask", "n_tok", "ids", "bias", "allowed")]
    assert epq_lib.epq_logits_adjust(x, *args, out=x) is x
    got = x.cpu().numpy()
    _same(got, _reference(**a))
    assert np.array_equal(got[1], a["x"][1]) and np.array_equal(got[2, 3:], a["x"][2, 3:])


def test_values(epq_lib):
    """Infinities, NaN and zeros: a masked NaN is -inf, -inf stays, a row that allows nothing is all -inf."""
    a = _inputs(1, 4, 100, 30, 4, seed=7)
    a["x"][0, :, 0], a["x"][0, :, 1], a["x"][0, :, 2], a["x"][0, :, 3] = math.nan, -math.inf, 0.0, -0.0
    a["x"][0, :, 90:] = math.nan
    a["allowed"][0, 1], a["allowed"][0, 2] = 0, -1
    a["bias"][0, 1] = -math.inf
    want = _reference(**a)[0]
    got = _run(epq_lib, **a)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.isneginf(got[0, 1]).all() and np.isnan(got[0, 2, 0]) and np.isnan(got[0, 2, 95])


def test_wide_rows(epq_lib):
    """Rows of a wider buffer through the C call, and no read of what lies between them."""
    import ctypes
    lib, O = epq_lib.load(), epq_lib._lib.LogitsOpts
    x, y = torch.randn(6, 1003, device="cuda"), torch.full((6, 1100), 7.0, device="cuda")
    pen, hist = torch.tensor([[1.5, 0.25, 0.5]] * 2, device="cuda"), torch.arange(0, 40, device="cuda").int().view(2, 20)
    o = O(penalties=pen.data_ptr(), history=hist.data_ptr(), max_history=20, ld=1003, out_ld=1100)
    assert lib.epq_logits_adjust(x.data_ptr(), 1000, 2, 3, ctypes.byref(o), y.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    want = epq_lib.epq_logits_adjust(x[:, :1000].contiguous().view(2, 3, 1000), pen, hist)
    assert torch.equal(y[:, :1000].reshape(2, 3, 1000), want) and (y[:, 1000:] == 7.0).all()


def test_many_rows_without_tokens(epq_lib):
    """More than a tree's rows, when no drafted tokens are named."""
    a = _inputs(2, 64, 700, 30, 3, seed=9, tree=False)
    x = np.concatenate([a["x"], a["x"][:, :30]], 1)
    got = _run(epq_lib, x, a["pen"], a["hist"], a["hlen"], a["plen"], ids=a["ids"], bias=a["bias"])
    _same(got, _reference(x, a["pen"], a["hist"], a["hlen"], a["plen"], ids=a["ids"], bias=a["bias"]))


def test_graph_and_verify(epq_lib):
    """Adjusted, then verified, as one step captured in a graph: no token that a grammar leaves out is accepted or drawn."""
    a = _inputs(2, 8, 3001, 40, 5, seed=11)
    a["n_tok"][:] = 8
    a["allowed"][:, :, 0] |= 6
    x = _gpu(a["x"])
    parent = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 3]] * 2, dtype=torch.int32, device="cuda")
    mask = epq_lib.epq_tree_mask(parent)
    u = torch.rand(2, 8, device="cuda")
    args = dict(penalties=_gpu(a["pen"]), history=_gpu(a["hist"]), tokens=_gpu(a["tokens"]), mask=mask, allowed=_gpu(a["allowed"]))
    out = torch.empty_like(x)
    ws = epq_lib.epq_verify_tree_workspace(x)

    def step():
        epq_lib.epq_logits_adjust(x, out=out, **args)
        return epq_lib.epq_verify_tree(out, args["tokens"], parent, u, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path, n, nxt, _ = step()
    bits = a["allowed"].view(np.uint32)
    for k in range(20):
        x.normal_(std=3.0)
        u.uniform_()
        graph.replay()
        for s in range(2):
            rows = path[s, : int(n[s])].tolist()
            toks = [int(a["tokens"][s, i]) for i in rows[1:]] + [int(nxt[s])]
            for row, t in zip(rows, toks):
                assert bits[s, row, t // 32] >> (t % 32) & 1


def test_many_sequences_and_empty_lists(epq_lib):
    """More sequences than a tree has tokens; histories and biases of no entries."""
    a = _inputs(300, 2, 70, 9, 3, seed=13)
    _same(_run(epq_lib, **a), _reference(**a))
    x = torch.randn(2, 3, 500, device="cuda")
    none = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    got = epq_lib.epq_logits_adjust(x, torch.full((2, 3), 2.0, device="cuda"), none, bias_ids=none, bias=none.float())
    assert torch.equal(got, x)


@pytest.mark.parametrize("r", [1e-12, 1e12, 3.0000002, 1e-3])
def test_quotients(epq_lib, r):
    """Logits from the smallest to the largest numbers over penalties of any size: the division's quotients."""
    rng = np.random.default_rng(5)
    n = 60000
    x = (2.0 ** rng.uniform(-140, 127, n) * rng.choice([-1.0, 1.0], n)).astype(F).reshape(1, 1, n)
    pen = np.array([[r, 0.0, 0.0]], dtype=F)
    hist = np.arange(n, dtype=np.int32).reshape(1, n)
    with np.errstate(all="ignore"):
        want = np.where(x > 0, x / F(r), x * F(r)).astype(F) - F(0)
    assert np.array_equal(_run(epq_lib, x, pen, hist), want)


def test_long_lists_in_one_chunk(epq_lib):
    """Lists longer than a CTA has threads, with drafted tokens among them, and just as long."""
    rng = np.random.default_rng(6)
    for m in (255, 256, 257, 600, 2048):
        hist = np.concatenate([rng.permutation(2048)[:m], np.full(20, 5)]).astype(np.int32).reshape(1, -1)
        x = rng.standard_normal((1, 8, 4000)).astype(F)
        tok = rng.integers(0, 2048, (1, 8)).astype(np.int32)
        tok[0, 3] = tok[0, 1]
        a = dict(x=x, pen=np.array([[1.7, 0.3, 0.2]], dtype=F), hist=hist, plen=np.array([m // 3], dtype=np.int32), tokens=tok,
                 ids=rng.integers(0, 4000, (1, 50)).astype(np.int32), bias=rng.standard_normal((1, 50)).astype(F))
        _same(_run(epq_lib, **a), _reference(**a))


def test_two_at_once(epq_lib):
    a, b = _inputs(4, 16, 9000, 500, 20, seed=15), _inputs(2, 5, 7001, 100, 3, seed=16)
    args = [[_gpu(c.get(k)) for k in ("x", "pen", "hist", "hlen", "plen", "tokens", "mask", "n_tok", "ids", "bias", "allowed")] for c in (a, b)]
    want = [epq_lib.epq_logits_adjust(*x) for x in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    got = [[epq_lib.epq_logits_adjust(*x, stream=st) for x, st in zip(args, streams)] for _ in range(8)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(p, w) for p, w in zip(pair, want))
