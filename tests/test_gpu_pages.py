"""GPU parity of epq_pages_* against the page-by-page oracle: tables, lengths,
reference counts and status exactly, and the bytes of every committed row."""
import random

import numpy as np
import pytest
import torch

from oracle import tree as T

pytestmark = pytest.mark.gpu


class Both:
    """The library's cache and the oracle's, driven together.  Oracle rows are
    tags; the library's rows are those tags as bytes in every layer, head and
    plane."""

    def __init__(self, epq, dev, layers=2, n_pages=24, kv=2, D=128, n_seq=4, max_pages=8, P=16):
        self.epq, self.dev = epq, dev
        self.c = epq.PagedKVCache(layers, n_pages, kv, D, n_seq, max_pages, P, dev)
        self.o = T.Pages(n_pages, n_seq, max_pages, P)
        self.n_seq, self.P, self.tag = n_seq, P, 0

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def row(self, tag, page_unit):
        """The bytes of a tagged row in one (layer, head, plane)."""
        rng = np.random.default_rng(tag * 1000 + page_unit)
        return rng.integers(0, 256, self.c.pool.shape[-1], dtype=np.uint8)

    def write(self, s, pos):
        """A new tagged row at a reserved position."""
        self.tag += 1
        page, slot = self.o.table[s][pos // self.P], pos % self.P
        self.o.rows[page, slot] = self.tag
        L, _, H, _, _, R = self.c.pool.shape
        b = np.stack([self.row(self.tag, u) for u in range(L * H * 2)]).reshape(L, H, 2, R)
        self.c.pool[:, page, :, :, slot] = torch.from_numpy(b).to(self.dev)

    def truncate(self, n):
        self.o.truncate(n)
        self.epq.epq_pages_truncate(self.c, self.i32(n))

    def fork(self, a, b):
        st = torch.full((len(a),), -7, dtype=torch.int32, device=self.dev)
        want = self.o.fork(a, b)
        self.epq.epq_pages_fork(self.c, self.i32(a), self.i32(b), st)
        assert st.tolist() == want
        return want

    def reserve(self, n):
        want = self.o.reserve(n)
        assert self.epq.epq_pages_reserve(self.c, self.i32(n)).tolist() == want
        return want

    def compact(self, path, keep):
        self.o.compact(path, keep)
        self.epq.epq_pages_compact(self.c, self.i32(path), self.i32(keep))

    def same(self):
        torch.cuda.synchronize()
        table = self.c.table.tolist()
        assert [[p for p in r if p >= 0] for r in table] == self.o.table
        assert all(r[len(t):] == [-1] * (len(r) - len(t)) for r, t in zip(table, self.o.table))
        assert self.c.length.tolist() == self.o.length and self.c.refs.tolist() == self.o.refs
        pool = self.c.pool.cpu().numpy()
        L, _, H, _, _, R = pool.shape
        for s in range(self.n_seq):
            for pos in range(self.o.length[s]):
                page, slot = self.o.table[s][pos // self.P], pos % self.P
                tag = self.o.rows[page, slot]
                got = pool[:, page, :, :, slot].reshape(L * H * 2, R)
                for u in (0, L * H * 2 - 1, tag % (L * H * 2)):
                    assert np.array_equal(got[u], self.row(tag, u)), (s, pos)
        assert self.epq.epq_device_error() == 0


@pytest.mark.parametrize("P, D", [(16, 128), (32, 256), (64, 128), (128, 128)])
def test_random_calls(epq_lib, cuda_dev, P, D):
    """Forks, truncations, reservations that fit or do not, and commits."""
    rnd = random.Random(P + D)
    n = 13
    b = Both(epq_lib, cuda_dev, D=D, P=P, n_pages=14, n_seq=4, max_pages=max(3, 96 // P))
    for step in range(60):
        op = rnd.randrange(5)
        if op == 0:
            k = rnd.randint(1, 3)
            b.fork([rnd.randint(-1, 4) for _ in range(k)], [rnd.randint(0, 4) for _ in range(k)])
        elif op == 1:
            b.truncate([rnd.choice([-1, -1, -1, rnd.randrange(90), 0]) for _ in range(4)])
        else:
            extra = [rnd.choice([n, n, 0, -1]) for _ in range(4)]
            ok = b.reserve(extra)
            path, keep = [[-1] * n for _ in range(4)], [0] * 4
            for s in range(4):
                if extra[s] <= 0 or ok[s] != 0:
                    continue
                for i in range(n):
                    b.write(s, b.o.length[s] + i)
                p = sorted(rnd.sample(range(n), rnd.randint(0, n)))
                path[s], keep[s] = p + [-1] * (n - len(p)), len(p)
            b.compact(path, keep)
        if step % 6 == 5:
            b.same()
    b.same()


def test_copy_on_write_rows_and_keeper(epq_lib, cuda_dev):
    """Three branches of one prompt: the first two copy the partly filled
    page, the last one keeps it; a full last page is shared for good."""
    b = Both(epq_lib, cuda_dev)
    assert b.reserve([21, 0, 0, 0]) == [0, 0, 0, 0]
    for i in range(21):
        b.write(0, i)
    b.compact([list(range(21)), [-1] * 21, [-1] * 21, [-1] * 21], [21, 0, 0, 0])
    assert b.fork([0, 0], [1, 2]) == [0, 0]
    b.same()
    assert b.reserve([3, 3, 3, 0]) == [0, 0, 0, 0]
    assert b.o.refs[1] == 1 and b.o.table[2][1] == 1 and b.o.refs[0] == 3
    b.same()
    b.truncate([16, 0, 0, -1])
    assert b.fork([0], [3]) == [0]
    assert b.reserve([1, 0, 0, 1]) == [0, 0, 0, 0]  # 16 positions fill their page: nothing is copied
    b.same()


def test_fork_refusals(epq_lib, cuda_dev):
    b = Both(epq_lib, cuda_dev)
    b.reserve([5, 0, 0, 0])
    for i in range(5):
        b.write(0, i)
    b.compact([list(range(5))] + [[-1] * 5] * 3, [5, 0, 0, 0])
    # the first entry names sequence 0 as a destination, so no entry may read it
    assert b.fork([0, 0, -1, 0, 0, 1], [0, 4, 2, 1, 1, 3]) == [1, 1, 1, 1, 1, 1]
    # out of range, done, twice the same, a source that is a destination
    assert b.fork([0, -1, 0, 0, 1], [4, 2, 1, 1, 3]) == [1, 1, 0, 1, 1]
    assert b.fork([0, 1], [1, 2]) == [1, 1]
    b.same()


def test_reserve_without_room(epq_lib, cuda_dev):
    """Pages run out: the first sequence that does not fit and all later ones
    stay as they are; one longer than its table is refused by itself."""
    b = Both(epq_lib, cuda_dev, n_pages=5, max_pages=4)
    assert b.reserve([20, 65, 40, 16]) == [0, 2, 0, 1]
    b.same()
    assert b.reserve([0, 1, 0, 0]) == [0, 1, 0, 0]
    b.truncate([0, -1, -1, -1])
    assert b.reserve([0, 32, 8, 1]) == [0, 0, 0, 1]
    b.same()


def test_reserve_many_pages(epq_lib, cuda_dev):
    """Free ids past one scan of the reference counts, and a long reservation."""
    b = Both(epq_lib, cuda_dev, layers=1, kv=1, n_pages=5000, n_seq=3, max_pages=3000, P=16)
    assert b.reserve([16 * 2049, 0, 5]) == [0, 0, 0]
    b.truncate([16 * 7, -1, -1])
    assert b.reserve([0, 16 * 2900, 16 * 30]) == [0, 0, 0]
    b.same()


def test_bad_state_is_not_followed(epq_lib, cuda_dev):
    """Page ids, lengths and path entries out of range: nothing is read or
    written through them, and a drafted row without a page is recorded."""
    c = epq_lib.PagedKVCache(1, 4, 1, 128, 2, 3, 16, cuda_dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    c.table.copy_(i32([[9, -5, 1 << 30], [0, 1, -1]]))
    c.length.copy_(i32([40, 1 << 30]))
    c.refs.copy_(i32([1, 1, 0, 0]))
    before = c.pool.clone()
    epq_lib.epq_pages_compact(c, i32([[0, 3, 2, 99], [1, 2, 3, -4]]), i32([4, 77]))
    torch.cuda.synchronize()
    assert torch.equal(before, c.pool) and c.length.tolist() == [44, 48]
    assert epq_lib.epq_device_error() == 5
    assert epq_lib.epq_pages_reserve(c, i32([2, 1])).tolist() == [0, 2]
    assert c.table.tolist() == [[9, -5, 2], [0, 1, -1]] and c.refs.tolist() == [1, 1, 1, 0]
    epq_lib.epq_pages_truncate(c, i32([0, 0]))
    assert c.refs.tolist() == [0, 0, 0, 0] and epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("P, D, rows", [(16, 128, 5), (64, 256, 63)])
def test_one_sequence_over_a_shared_page(epq_lib, cuda_dev, P, D, rows):
    """Two caches over one pool and its reference counts, the second with a
    single sequence: its partly filled page, which the first holds too, is
    copied before it is written."""
    b = Both(epq_lib, cuda_dev, D=D, P=P)
    b.reserve([rows, 0, 0, 0])
    for i in range(rows):
        b.write(0, i)
    b.compact([list(range(rows))] + [[-1] * rows] * 3, [rows, 0, 0, 0])
    b.same()
    shared = b.o.table[0][0]
    b.c.refs[shared] += 1
    one = epq_lib.PagedKVCache.over(b.c.pool, b.c.table[:1].clone(), b.c.length[:1].clone(), b.c.refs)
    kept = b.c.pool[:, shared].clone()
    assert epq_lib.epq_pages_reserve(one, b.i32([1])).tolist() == [0]
    own = one.table[0, 0].item()
    assert own != shared and b.c.refs.tolist()[shared] == b.c.refs.tolist()[own] == 1
    assert torch.equal(b.c.pool[:, own, :, :, :rows], kept[:, :, :, :rows])
    assert torch.equal(b.c.pool[:, shared], kept)
    assert epq_lib.epq_device_error() == 0


def test_copy_past_32_bits(epq_lib, cuda_dev):
    """The only free pages lie more than 2^32 bytes into the pool."""
    c = epq_lib.PagedKVCache(2, 17000, 8, 128, 2, 4, 128, cuda_dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    c.refs[:16990] = 1
    assert epq_lib.epq_pages_reserve(c, i32([9, 0])).tolist() == [0, 0] and c.table[0, 0].item() == 16990
    c.pool[:, 16990, :, :, :9] = torch.randint(0, 256, c.pool[:, 0, :, :, :9].shape, dtype=torch.uint8, device=cuda_dev)
    c.length[0] = 9
    epq_lib.epq_pages_fork(c, i32([0]), i32([1]))
    assert epq_lib.epq_pages_reserve(c, i32([0, 3])).tolist() == [0, 0] and c.table[1, 0].item() == 16991
    assert torch.equal(c.pool[:, 16991, :, :, :9], c.pool[:, 16990, :, :, :9]) and not c.pool[:, 16992].any()
    assert epq_lib.epq_device_error() == 0


def test_results_of_a_call_on_another_stream(epq_lib, cuda_dev):
    """What a call on another stream allocates for its results is memory that no earlier work of the current stream can
    still be using, and is given out again, once the caller drops it, only after both streams are done with it."""
    cache = epq_lib.PagedKVCache(1, 4, 1, 128, 3, 2, 16, cuda_dev)
    extra = torch.ones(3, dtype=torch.int32, device=cuda_dev)
    parent = torch.full((3, 2), -1, dtype=torch.int32, device=cuda_dev)
    q, kv = (torch.zeros((3, 2, 128), device=cuda_dev) for _ in range(2))
    logits, u = torch.zeros((3, 2, 100), device=cuda_dev), torch.zeros((3, 2), device=cuda_dev)
    calls = [lambda s: [epq_lib.epq_pages_reserve(cache, extra, stream=s)],
             lambda s: [epq_lib.epq_tree_mask(parent, stream=s)],
             lambda s: [epq_lib.epq_attention_tree(q, kv, kv, cache, 0, 1, 1.0, stream=s)],
             lambda s: list(epq_lib.epq_verify_tree(logits, parent, parent, u, stream=s))]

    def wait():
        torch.cuda._sleep(200_000_000)  # about 0.1 s

    def again(like, stream):
        """Where the next tensors of these shapes and of this stream's memory lie."""
        with torch.cuda.stream(stream):
            fresh = [torch.empty(r[0], dtype=r[1], device=cuda_dev) for r in like for _ in range(4)]
            return {f.data_ptr() for f in fresh}

    here = torch.cuda.current_stream()
    for call in calls:
        results = call(None)
        like = [(r.shape, r.dtype) for r in results]
        results.clear()  # memory that the call below could be given
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for s in (side, side.cuda_stream):
            before = again(like, here)
            with torch.cuda.stream(side):
                wait()
            results = call(s)
            at = {r.data_ptr() for r in results}
            assert not at & before
            results.clear()  # while `side` has yet to write them
            assert not again(like, here) & at
            torch.cuda.synchronize()
            results = call(s)
            at = {r.data_ptr() for r in results}
            here.wait_stream(side)
            wait()  # the current stream reads them
            results.clear()
            with torch.cuda.stream(side):
                wait()
            assert not again(like, side) & at
            torch.cuda.synchronize()
    assert epq_lib.epq_device_error() == 0


def test_step_of_sequences_without_room(epq_lib, cuda_dev):
    """The step of the usage text: two branches of one page and no free one, next to a sequence with room.  The branches
    sit it out, their shared page keeps its bytes, and their next tokens are -1."""
    cache = epq_lib.PagedKVCache(2, 3, 2, 128, 3, 4, 16, cuda_dev)
    cache.pool.copy_(torch.randint(0, 64, cache.pool.shape, dtype=torch.uint8, device=cuda_dev))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)  # noqa: E731
    epq_lib.epq_pages_reserve(cache, i32(20, 0, 10))  # all three pages
    cache.length.copy_(i32(20, 0, 10))
    epq_lib.epq_pages_fork(cache, i32(0), i32(1))
    before = cache.pool.clone()
    extra = i32(4, 4, 4)
    parent = i32(-1, 0, 1, 2).repeat(3, 1)
    q, k, v = (torch.randn((3, 4, n * 128), device=cuda_dev) for n in (4, 2, 2))
    logits, u = torch.randn((3, 4, 50), device=cuda_dev), torch.zeros((3, 4), device=cuda_dev)
    order = [2, 0, 1]  # the sequence with room first: later ones do not fit
    cache.table.copy_(cache.table[order].clone())
    cache.length.copy_(cache.length[order].clone())
    status = epq_lib.epq_pages_reserve(cache, extra)
    n_tok = extra * (status == 0)
    mask = epq_lib.epq_tree_mask(parent)
    for layer in range(2):
        epq_lib.epq_attention_tree(q, k, v, cache, layer, 4, 0.1, mask=mask, n_tok=n_tok)
    path, n, nxt, _ = epq_lib.epq_verify_tree(logits, parent.clamp(min=0), parent, u, n_tok=n_tok)
    epq_lib.epq_pages_compact(cache, path, n)
    assert status.tolist() == [0, 1, 1] and n_tok.tolist() == [4, 0, 0]
    assert n.tolist()[1:] == [0, 0] and nxt.tolist()[1:] == [-1, -1] and n[0].item() >= 1
    assert cache.length.tolist() == [10 + n[0].item(), 20, 20]
    own = cache.table[0, 0].item()
    others = [p for p in range(3) if p != own]
    assert torch.equal(cache.pool[:, others], before[:, others]) and not torch.equal(cache.pool[:, own], before[:, own])
    assert epq_lib.epq_device_error() == 0
