"""GPU parity of epq_verify_tree and epq_tree_mask against the float64 oracle:
paths, counts and next tokens exactly (a wrong side of a comparison needs u
within about 1e-7 of a threshold), the log sums within their rounding."""
import numpy as np
import pytest
import torch

from oracle import tree as T

pytestmark = pytest.mark.gpu


def _tree(rng, n):
    return [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]


def _case(seed, nseq, ntok, vocab, temperature, draft, noise=0.5, spread=3.0):
    rng = np.random.default_rng(seed)
    logits = (spread * rng.standard_normal((nseq, ntok, vocab))).astype(np.float32)
    parent = np.array([_tree(rng, ntok) for _ in range(nseq)], np.int32)
    z = logits + noise * rng.standard_normal(logits.shape)
    q = np.exp((z - z.max(-1, keepdims=True)) / (temperature or 1.0))
    q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.zeros((nseq, ntok), np.int32)
    for s in range(nseq):
        for i in range(1, ntok):
            p = q[s, parent[s, i]].astype(np.float64)
            tokens[s, i] = rng.choice(vocab, p=p / p.sum())
    u = rng.random((nseq, ntok)).astype(np.float32)
    return logits, tokens, parent, np.minimum(u, np.float32(1 - 2.0 ** -24)), q if draft else None


def _check(epq, dev, case, temperature, n_tok=None):
    logits, tokens, parent, u, q = case
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    nt = None if n_tok is None else torch.tensor(n_tok, dtype=torch.int32, device=dev)
    ws = epq.epq_verify_tree_workspace(t(logits))
    got = [x.cpu().numpy() for x in epq.epq_verify_tree(t(logits), t(tokens), t(parent), t(u), draft=t(q), n_tok=nt,
                                                        temperature=temperature, workspace=ws)]
    again = [x.cpu().numpy() for x in epq.epq_verify_tree(t(logits), t(tokens), t(parent), t(u), draft=t(q), n_tok=nt,
                                                          temperature=temperature, workspace=ws)]
    assert all(np.array_equal(a, b) for a, b in zip(got, again))
    path, count, nxt, lse = got
    nseq, ntok, vocab = logits.shape
    for s in range(nseq):
        n = ntok if n_tok is None else n_tok[s]
        if n == 0:
            assert count[s] == 0 and nxt[s] == -1 and (path[s] == -1).all() and (lse[s] == 0).all()
            continue
        wp, wn, wl = T.verify_tree(logits[s, :n], tokens[s, :n], parent[s, :n], u[s, :n], None if q is None else q[s, :n],
                                   temperature)
        assert path[s].tolist() == wp + [-1] * (ntok - len(wp)), s
        assert count[s] == len(wp) and nxt[s] == wn, s
        # log of a float32 sum of up to vocab terms, each through at most vocab/256 + 32 additions; the argument
        # (l - max) / T is off by three roundings of its size
        tol = (vocab / 256 + 64) * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(wl).max() + np.ptp(logits[s]) / (temperature or 1.0))
        assert np.abs(lse[s, :n] - wl).max() <= tol and (lse[s, n:] == 0).all()
    return path, count, nxt


@pytest.mark.parametrize("vocab", [1, 2, 31, 1000, 4097, 50001, 128256])
@pytest.mark.parametrize("draft", [False, True])
def test_sizes(epq_lib, cuda_dev, vocab, draft):
    nseq, ntok = (3, 9) if vocab <= 5000 else (2, 5)
    for k, temperature in enumerate((1.0, 0.0, 0.7)):
        _check(epq_lib, cuda_dev, _case(vocab + k, nseq, ntok, vocab, temperature, draft), temperature)


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_many_walks(epq_lib, cuda_dev, draft, seed):
    """Wide trees, both far and near drafts: rejections among siblings, long paths, ends at every depth."""
    _, count, _ = _check(epq_lib, cuda_dev, _case(seed, 24, 64, 97, 1.3, draft, noise=(0.1, 3.0)[seed % 2]), 1.3)
    if draft and seed % 2 == 0:  # near drafts: paths of several lengths
        assert count.max() > 2 and len(set(count.tolist())) > 2


@pytest.mark.parametrize("ntok", [1, 2, 64])
def test_ragged_trees(epq_lib, cuda_dev, ntok):
    n_tok = [0, 1, ntok, max(1, ntok // 2)]
    for temperature in (0.0, 1.0):
        _check(epq_lib, cuda_dev, _case(ntok, 4, ntok, 3001, temperature, True), temperature, n_tok)


def test_excluded_tokens_and_ids_out_of_range(epq_lib, cuda_dev):
    logits, tokens, parent, u, q = _case(11, 4, 8, 600, 1.0, False)
    logits[:, :, 100:] = -np.inf
    logits[1, :, :] = -np.inf
    logits[1, :, 599] = -3.0  # one token left
    tokens[0, 1:4] = [-1, 600, 2 ** 31 - 1]
    tokens[2, 1:3] = [250, 599]  # excluded by the target
    u[3, :] = 0.0
    _check(epq_lib, cuda_dev, (logits, tokens, parent, u, None), 1.0)
    _check(epq_lib, cuda_dev, (logits, tokens, parent, u, None), 0.0)
    u[:] = np.float32(1 - 2.0 ** -24)
    _check(epq_lib, cuda_dev, (logits, tokens, parent, u, None), 1.0)


def test_draft_equal_to_the_target_is_accepted(epq_lib, cuda_dev):
    """q = p: every first child is accepted; rejected siblings cannot occur on the way."""
    case = _case(21, 8, 12, 500, 1.0, True, noise=0.0)
    case[2][:] = np.arange(-1, 11)  # chains
    case[3][:] = np.minimum(case[3], 0.999)
    path, count, _ = _check(epq_lib, cuda_dev, case, 1.0)
    assert (count == 12).all()


def test_siblings_drawn_twice(epq_lib, cuda_dev):
    logits, tokens, parent, u, q = _case(31, 6, 10, 50, 1.0, True, noise=2.0)
    parent[:, 1:] = 0
    tokens[:, 5:] = tokens[:, 1:6]
    _check(epq_lib, cuda_dev, (logits, tokens, parent, u, q), 1.0)
    _check(epq_lib, cuda_dev, (logits, tokens, parent, u, None), 1.0)


def test_row_strides(epq_lib, cuda_dev):
    """Rows further apart than the vocabulary, through the C entry."""
    import ctypes

    logits, tokens, parent, u, q = _case(41, 2, 5, 777, 1.0, True)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)  # noqa: E731
    wide = torch.full((2, 5, 1001), float("nan"), device=cuda_dev)
    wide[..., :777] = t(logits)
    qw = torch.full((2, 5, 801), float("nan"), device=cuda_dev)
    qw[..., :777] = t(q)
    ws = torch.zeros(4096, dtype=torch.uint8, device=cuda_dev)
    path, na, nx = (torch.empty(n, dtype=torch.int32, device=cuda_dev) for n in ((2, 5), (2,), (2,)))
    tt, tp, tu = t(tokens), t(parent), t(u)
    lib = epq_lib.load()
    from moe_experts_gb300 import _lib as L
    o = L.VerifyOpts(qw.data_ptr(), None, 1.0, 1001, 801)
    p = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    assert ws.numel() >= lib.epq_verify_tree_workspace_bytes(2, 5, 777)
    assert lib.epq_verify_tree(p(wide), 777, p(tt), p(tp), p(tu), 2, 5, ctypes.byref(o), p(path), p(na), p(nx), None, p(ws),
                               ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    for s in range(2):
        wp, wn, _ = T.verify_tree(logits[s], tokens[s], parent[s], u[s], q[s], 1.0)
        assert path[s, :len(wp)].tolist() == wp and na[s].item() == len(wp) and nx[s].item() == wn


def test_tree_mask(epq_lib, cuda_dev):
    rng = np.random.default_rng(2)
    for n in (1, 2, 33, 64):
        parent = np.array([_tree(rng, n) for _ in range(5)], np.int32)
        parent[1] = np.arange(-1, n - 1)
        parent[2, rng.integers(0, n)] = 77
        got = epq_lib.epq_tree_mask(torch.from_numpy(parent).to(cuda_dev)).cpu().numpy().view(np.uint64)
        assert [[int(m) for m in r] for r in got] == [T.ancestors(p) for p in parent.tolist()]


def _one(epq, dev, logits, tokens, parent, u, q=None, temperature=1.0):
    """(path, next token) of one sequence."""
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(np.asarray(a, d)[None])).to(dev)  # noqa: E731
    nxt = torch.full((1,), -7, dtype=torch.int32, device=dev)
    path, n, _, _ = epq.epq_verify_tree(t(logits, np.float32), t(tokens, np.int32), t(parent, np.int32), t(u, np.float32),
                                        draft=None if q is None else t(q, np.float32), temperature=temperature, next_token=nxt)
    return path[0, :n.item()].tolist(), nxt.item()


@pytest.mark.parametrize("vocab", [500, 128256])
@pytest.mark.parametrize("temperature", [1.0, 0.05])
def test_weights_below_half_a_unit(epq_lib, cuda_dev, vocab, temperature):
    """Logits more than 45 ln 2 = 31.2 (times the temperature) below the largest weigh nothing: where only they are
    left, nothing is left, and the state before stands."""
    rng = np.random.default_rng(vocab)
    logits = np.zeros((2, vocab))
    far = rng.random(vocab) < 0.9
    far[:4] = False
    logits[:, ~far] = -20.0 - 5.0 * rng.random((~far).sum())
    logits[:, far] = -31.3 - 13.0 * rng.random(far.sum())  # to 44.3: to 64 ln 2
    logits[:, :4] = 0.0
    logits = (logits * temperature).astype(np.float32)
    q = np.zeros((2, vocab), np.float32)
    q[:, :4] = 0.2501
    q[:, ~far] = np.maximum(q[:, ~far], np.float32(1e-5))  # more than the target has
    without = np.where(far, -np.inf, logits)
    for u0 in (0.0, 0.3, 0.6, 0.9):
        u = np.array([u0, 0.99999], np.float32)
        want = T.verify_tree(without, [0, 2], [-1, 0], u, q, temperature)
        assert want[0] == [0] and want[1] < 4
        assert _one(epq_lib, cuda_dev, logits, [0, 2], [-1, 0], u, q, temperature) == (want[0], want[1])


@pytest.mark.parametrize("seed", range(12))
def test_siblings_after_a_dominating_one(epq_lib, cuda_dev, seed):
    """Given children that hold nearly all the mass: after the first is rejected, the others are judged by what is left,
    whatever part of the whole it is.  Weights are held in units of 2^-44 of the largest, of which the rest's have about
    170 each: the walk that is expected has the weights in these units."""
    rng = np.random.default_rng(seed)
    vocab, n = 128256, 4
    rest = rng.random(vocab) * 10.0 ** rng.uniform(-11, -10)  # about 1e-6 to 6e-6 in all
    logits = np.log(rest)
    a, b, c = rng.choice(vocab, 3, replace=False)
    logits[a] = 0.0
    logits[b], logits[c] = np.log(rest.sum() * 0.5), np.log(rest.sum() * 0.3)
    logits = np.tile(logits.astype(np.float32), (n, 1))
    w = np.exp(logits[0].astype(np.float64))
    with np.errstate(divide="ignore"):
        held = np.tile(np.log(np.rint(w * 2.0 ** 44) * 2.0 ** -44), (n, 1))
    left = w.sum() - w[a]
    for near in (-1e-3, -1e-5, 1e-5, 1e-3):
        for second in (b, c):
            third = c if second == b else b
            for u2, u3 in ((w[second] / left * (1 + near), 0.0), (0.999999, w[third] / (left - w[second]) * (1 + near))):
                u = np.array([0.4, 1 - 2.0 ** -23, u2, u3], np.float32)
                want = T.verify_tree(held, [0, a, second, third], [-1, 0, 0, 0], u)
                assert len(want[0]) == 1 or want[0][1] > 1
                assert _one(epq_lib, cuda_dev, logits, [0, a, second, third], [-1, 0, 0, 0], u) == (want[0], want[1])


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("spread", [0.5, 3.0, 8.0])
def test_next_to_a_threshold(epq_lib, cuda_dev, draft, spread):
    """The two float32 u on either side of an acceptance's border: accepted and not.  (Weights are good to 2^-29 = 1.9e-9
    of themselves: a border that close to u is left out.)"""
    rng = np.random.default_rng(int(10 * spread))
    vocab, nseq, temperature = 50001, 64, float(np.float32(0.7))  # as the call takes it
    logits = (spread * rng.standard_normal((nseq, 2, vocab))).astype(np.float32)
    order = logits[:, 0].argsort(1)
    x = order[np.arange(nseq), -1 - np.arange(nseq) % 8].astype(np.int32)
    z = logits.astype(np.float64) / temperature
    w = np.exp(z - z.max(-1, keepdims=True))
    at = (w[np.arange(nseq), 0, x] / w[:, 0].sum(1))
    q = None
    if draft:
        q = (np.exp(0.3 * rng.standard_normal(logits.shape)) * w / w.sum(-1, keepdims=True)).astype(np.float32)
        at = at / q[np.arange(nseq), 0, x].astype(np.float64)
    lo = at.astype(np.float32)
    lo = np.where(lo.astype(np.float64) < at, lo, np.nextafter(lo, np.float32(0)))
    hi = np.nextafter(lo, np.float32(1))
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(np.asarray(a, d))).to(cuda_dev)  # noqa: E731
    judged = 0
    for u, want in ((lo, 2), (hi, 1)):
        uu = np.stack([np.full(nseq, 0.5), u], 1)
        n = epq_lib.epq_verify_tree(t(logits, np.float32), t(np.stack([x * 0, x], 1), np.int32), t([[-1, 0]] * nseq, np.int32),
                                    t(uu, np.float32), draft=None if q is None else t(q, np.float32),
                                    temperature=temperature)[1].cpu().numpy()
        clear = (np.abs(u.astype(np.float64) / at - 1) > 4 * 2.0 ** -29) & (u < 1) & (u > 0)
        judged += clear.sum()
        assert (n[clear] == want).all(), np.flatnonzero(clear & (n != want))
    assert judged > nseq / 2


@pytest.mark.parametrize("draft", [False, True])
def test_random_numbers_outside_their_range(epq_lib, cuda_dev, draft):
    """u outside [0, 1) is the nearest number in it, NaN is 0: a next token is always written."""
    logits, tokens, parent, u, q = _case(51, 1, 5, 700, 1.0, draft)
    last = 1 - 2.0 ** -24
    for bad, good in ((1.0, last), (1e30, last), (np.inf, last), (-0.5, 0.0), (-np.inf, 0.0), (np.nan, 0.0)):
        for where in ([0], [0, 1, 2, 3, 4]):
            ub, ug = u[0].copy(), u[0].copy()
            ub[where], ug[where] = bad, good
            want = T.verify_tree(logits[0], tokens[0], parent[0], ug, None if q is None else q[0])
            got = _one(epq_lib, cuda_dev, logits[0], tokens[0], parent[0], ub, None if q is None else q[0])
            assert got == (want[0], want[1]), (bad, where)


@pytest.mark.parametrize("draft", [False, True])
def test_logits_that_are_nan_are_excluded(epq_lib, cuda_dev, draft):
    """A NaN logit weighs nothing, as -inf does: the same path and next token (the row's log sum is NaN)."""
    for seed in range(8):
        logits, tokens, parent, u, q = _case(60 + seed, 1, 6, 900, 1.0, draft)
        rng = np.random.default_rng(seed)
        bad = rng.random(logits.shape) < 0.05
        if seed % 2:
            bad[0, parent[0, 1], tokens[0, 1]] = True  # a drafted token among them
        without = np.where(bad, -np.inf, logits).astype(np.float32)
        want = T.verify_tree(without[0], tokens[0], parent[0], u[0], None if q is None else q[0])
        got = _one(epq_lib, cuda_dev, np.where(bad, np.nan, logits)[0], tokens[0], parent[0], u[0], None if q is None else q[0])
        assert got == (want[0], want[1]), seed


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("temperature", [1e-30, 1e-40, 1e30])
def test_extreme_temperatures(epq_lib, cuda_dev, draft, temperature):
    """The largest logit has all the weight, or every token the same."""
    for seed in range(4):
        logits, tokens, parent, u, q = _case(80 + seed, 1, 6, 700, 1.0, draft)
        top = logits[0].argmax(1)
        tokens[0, 1:] = np.where(seed % 2 + np.arange(1, 6) % 2 > 0, top[parent[0, 1:]], tokens[0, 1:])
        want = T.verify_tree(logits[0], tokens[0], parent[0], u[0], None if q is None else q[0], temperature)
        got = _one(epq_lib, cuda_dev, logits[0], tokens[0], parent[0], u[0], None if q is None else q[0], temperature)
        assert got == (want[0], want[1]), seed


def test_logits_and_draft_from_any_float(epq_lib, cuda_dev):
    """Rows that begin between two 16-byte boundaries: a view into a larger tensor."""
    for shift in (1, 2, 3):
        logits, tokens, parent, u, q = _case(70 + shift, 2, 5, 1001, 1.0, True)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(cuda_dev)  # noqa: E731

        def moved(a):
            wide = torch.full((a.size + 8,), float("nan"), device=cuda_dev)
            wide[shift:shift + a.size] = t(a).reshape(-1)
            return wide[shift:shift + a.size].view(a.shape)

        got = epq_lib.epq_verify_tree(moved(logits), t(tokens), t(parent), t(u), draft=moved(q))
        want = epq_lib.epq_verify_tree(t(logits), t(tokens), t(parent), t(u), draft=t(q))
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        assert torch.equal(got[3], want[3]) or torch.allclose(got[3], want[3], rtol=0, atol=1e-5)
