"""CPU pins of the tree-verification oracle (oracle/tree.py): closed forms of
masks and attention, the acceptance rule's output distribution, and the page
bookkeeping's invariants."""
import itertools
import random

import numpy as np
import pytest

from oracle import tree as T


def test_ancestors_of_a_chain_and_a_fan():
    assert T.ancestors([-1, 0, 1, 2]) == [1, 3, 7, 15]
    assert T.ancestors([-1, 0, 0, 2, 5]) == [1, 3, 5, 13, 16]  # a parent after its child starts a tree of its own


def test_attention_closed_forms():
    K, V = np.zeros((3, 4)), np.arange(12.0).reshape(3, 4)
    q = np.zeros((2, 4))
    out, _, _ = T.tree_attention_f64(q, K, V, 1, [1, 2], 1.0)  # equal scores: the mean of what a token sees
    assert np.allclose(out[0], (V[0] + V[1]) / 2) and np.allclose(out[1], (V[0] + V[2]) / 2)
    K[1, 0], q[0, 0] = 1.0, np.log(3.0)
    out, _, _ = T.tree_attention_f64(q, K, V, 1, [1, 0], 1.0)
    assert np.allclose(out[0], V[0] / 4 + 3 * V[1] / 4) and np.allclose(out[1], V[0])
    out, _, _ = T.tree_attention_f64(q, K[1:], V[1:], 0, [0, 2], 1.0)  # nothing seen: 0
    assert np.array_equal(out[0], np.zeros(4))


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("parent", [[-1, 0], [-1, 0, 0], [-1, 0, 1]])
def test_first_token_has_the_targets_distribution(draft, parent):
    """Over all drafted tokens (weighted by the draft's probabilities) and a
    grid of u, the first kept token is distributed as the target."""
    rng = np.random.default_rng(3)
    V, n, grid = 3, len(parent), 24
    logits = rng.standard_normal((n, V))
    q = rng.dirichlet(np.ones(V), n)
    us = (np.arange(grid) + 0.5) / grid
    got = np.zeros(V)
    for tok in itertools.product(range(V), repeat=n - 1):
        weight = np.prod([q[parent[i + 1]][t] for i, t in enumerate(tok)]) if draft else float(tok == (1, 2)[: n - 1])
        if weight == 0.0:
            continue
        for u in itertools.product(us, repeat=n):
            path, nxt, _ = T.verify_tree(logits, (0, *tok), parent, u, q if draft else None)
            got[tok[path[1] - 1] if len(path) > 1 else nxt] += weight / grid ** n
    want = np.exp(logits[0]) / np.exp(logits[0]).sum()
    # a grid of cells of 1/grid misses a threshold by at most half a cell: at most one for each of n comparisons
    assert np.abs(got - want).max() <= n * 0.5 / grid + 1e-9


def test_greedy_takes_the_first_largest_logit():
    logits = np.array([[0.0, 2.0, 2.0], [1.0, 0.0, 0.0], [0.0, 0.0, 5.0]])
    assert T.verify_tree(logits, [0, 2, 1], [-1, 0, 0], None, temperature=0)[:2] == ([0, 2], 2)
    assert T.verify_tree(logits, [0, 1, 1], [-1, 0, 1], None, temperature=0)[:2] == ([0, 1], 0)


def test_pages_invariants():
    """Random calls: refs count the holders, no two sequences write one page,
    and every sequence reads back what was written to it."""
    rnd = random.Random(5)
    p = T.Pages(14, 5, 6, 4)
    want = [[] for _ in range(5)]
    for step in range(400):
        op = rnd.randrange(4)
        if op == 0:
            a, b = rnd.randrange(5), rnd.randrange(5)
            if p.fork([a], [b]) == [0]:
                want[b] = list(want[a])
        elif op == 1:
            cut = [rnd.choice([-1, -1, rnd.randrange(20), 0]) for _ in range(5)]
            p.truncate(cut)
            want = [w if n < 0 else w[:n] for w, n in zip(want, cut)]
        else:
            n = 5
            ok = p.reserve([n if rnd.random() < 0.7 else 0 for _ in range(5)])
            ext = [s for s in range(5) if ok[s] == 0 and len(p.table[s]) * 4 >= p.length[s] + n]
            keep, path = [0] * 5, [[-1] * n for _ in range(5)]
            for s in ext:
                first = p.table[s][p.length[s] // 4]
                if p.refs[first] > 1:
                    continue
                for i in range(n):
                    at = p.length[s] + i
                    p.rows[p.table[s][at // 4], at % 4] = (step, s, i)
                path[s] = sorted(rnd.sample(range(n), rnd.randint(1, n)))
                keep[s] = len(path[s])
                path[s] += [-1] * (n - keep[s])
                want[s] = want[s] + [(step, s, i) for i in path[s] if i >= 0]
            p.compact(path, keep)
        held = [page for t in p.table for page in t]
        assert [held.count(i) for i in range(14)] == p.refs
        for s in range(5):
            assert p.length[s] == len(want[s])
            assert [p.rows[p.table[s][i // 4], i % 4] for i in range(p.length[s])] == want[s]
