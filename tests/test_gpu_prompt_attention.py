"""GPU parity of epq_attention_prompt against the formula in 64 bits, within
bounds that count float32 roundings: a score is off by at most ds = (32 + D/4)
2^-24 scale sum |q||k| (D/4 additions of a dot product that pass through one
accumulator, 32 for the rest: the parts of an operand, the scale, the
exponential's argument), which changes a weight by a factor within exp(+-2 ds);
a sum over T positions is off by (32 + T/4) 2^-24 of the sum of magnitudes.

Weights have a floor besides.  The kernel holds a weight w (1 at the row's
maximum) as two halves of w' = 2^15 w: the 11 leading bits, and the rest
rounded.  A half is a multiple of 2^-24, so where w' is small each of the two
roundings is off by up to 2^-25, whatever w' is: 2^-24 of w', 2^-39 of w.  An
output is off by up to 2^-39 sum_j |v_j| for it, which shows where every larger
weight meets a value of 0."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F64 = torch.float64


def _rows(x):
    """float32 [..., D] -> cache rows in bytes (what a row holds is all that matters here)."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    d = (b.abs().amax(-1, keepdim=True) / 127).half()
    f = d.float()
    c = torch.where(f == 0, 0.0, (b / torch.where(f == 0, 1.0, f)).round().clamp(-127, 127)).to(torch.int8)
    return torch.cat([d[..., 0].contiguous().view(torch.uint8), c.view(torch.uint8).reshape(x.shape)], -1)


def _values(rows):
    D = rows.shape[-1] * 16 // 17
    f = rows[..., : D // 16].contiguous().view(torch.float16).double().repeat_interleave(32, -1)
    return f * rows[..., D // 16:].contiguous().view(torch.int8).double()


class Case:
    def __init__(self, epq, lengths, n_tok, heads, kv, D, P, window=0, seed=0, layers=1, layer=0, spread=2.0, ntok=None, kmul=1.0, vmul=1.0, qmul=1.0):
        self.epq, self.lengths, self.n_tok, self.heads, self.kv, self.D, self.P = epq, lengths, n_tok, heads, kv, D, P
        self.window, self.layer, self.ntok = window, layer, max(n_tok) if ntok is None else ntok
        g = self.g = torch.Generator(device="cuda").manual_seed(seed * 1009 + sum(lengths) + 7 * sum(n_tok) + D + P)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        each = [-(-(n + t) // P) for n, t in zip(lengths, n_tok)]
        n_pages = sum(each) + 2
        self.c = epq.PagedKVCache(layers, n_pages, kv, D, len(lengths), max(max(each), 1) + 1, P)
        # what no position holds: rows whose factors are NaN, with random codes
        self.c.pool.copy_(torch.randint(0, 256, self.c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
        self.c.pool[..., : D // 16].view(torch.float16)[:] = math.nan
        ids, at = torch.randperm(n_pages, generator=g, device="cuda").int(), 0
        for s, n in enumerate(each):
            self.c.table[s, :n] = ids[at:at + n]
            at += n
            T = lengths[s] + n_tok[s]
            x = rand(T, kv, 2, D)
            x[:, :, 0] *= kmul
            x[:, :, 1] *= vmul
            if T:
                self.put(s, torch.arange(T, device="cuda"), _rows(x))
        self.c.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        self.q = rand(len(lengths), self.ntok, heads * D) * spread * qmul
        for s, t in enumerate(n_tok):
            self.q[s, t:] = math.nan  # not read
        self.scale = 1 / math.sqrt(D)
        if not isinstance(kmul, torch.Tensor):
            self.scale /= qmul * kmul

    def put(self, s, pos, rows):
        """rows [positions, kv, 2, row] at positions of a sequence."""
        self.c.pool[self.layer, self.c.table[s].long()[pos // self.P], :, :, pos % self.P] = rows

    def rows(self, s):
        pos = torch.arange(self.lengths[s] + self.n_tok[s], device="cuda")
        return self.c.pool[self.layer, self.c.table[s].long()[pos // self.P], :, :, pos % self.P]

    def run(self, q=None, **kw):
        nt = torch.tensor(self.n_tok, dtype=torch.int32, device="cuda")
        return self.epq.epq_attention_prompt(self.q if q is None else q, self.c, self.layer, self.heads, self.scale, window=self.window, n_tok=nt, **kw)

    def check(self, out=None, hidden=None, **kw):
        """hidden: positions of each sequence that are left out."""
        if out is None:
            out = self.run(**kw)
        D, G = self.D, self.heads // self.kv
        got = out.view(len(self.lengths), self.ntok, self.heads, D).double()
        for s, (n, t) in enumerate(zip(self.lengths, self.n_tok)):
            assert not got[s, t:].any()
            if t == 0:
                continue
            behind = n + torch.arange(t, device="cuda")[:, None] - torch.arange(n + t, device="cuda")
            see = (behind >= 0) & ((behind < self.window) if self.window else True)
            if hidden is not None:
                see[:, hidden[s]] = False
            x = _values(self.rows(s))  # [T, kv, 2, D]
            lost = ~torch.isfinite(x).all(-1).all(-1)  # [T, kv]: a factor is not finite
            x = torch.where(torch.isfinite(x), x, 0.0)
            for h in range(self.kv):
                K, V = x[:, h, 0], x[:, h, 1]
                q = self.q[s, :t].view(t, self.heads, D)[:, h * G:(h + 1) * G].double()
                sc = (q @ K.T * self.scale).masked_fill(~see[:, None], -math.inf)
                smag = (q.abs() @ K.abs().T * self.scale).masked_fill(~see[:, None], 0.0).amax(-1)
                w = torch.softmax(sc, -1).nan_to_num(0.0)
                ds = (32 + D / 4) * 2.0 ** -24 * smag[..., None]
                bound = (w @ V.abs()) * (torch.expm1(2 * ds) + 2 * (32 + (n + t) / 4) * 2.0 ** -24)
                bound = bound + 2.0 ** -39 * V.abs().sum(0) + 1e-30
                out_h = got[s, :t, h * G:(h + 1) * G]
                nan = (see & lost[:, h]).any(1)
                assert torch.isnan(out_h[nan]).all()
                off = torch.where(nan[:, None, None], 0.0, (out_h - w @ V).abs() / bound)
                assert (off <= 1).all(), f"seq {s} head {h}: {off.max().item():.3g} at {(off == off.max()).nonzero()[0].tolist()}"
        return out


SHAPES = [
    # lengths, n_tok, heads, kv, D, page, window
    ([0], [1], 1, 1, 128, 16, 0),
    ([0], [65], 32, 8, 128, 64, 0),
    ([37], [1], 32, 8, 128, 64, 0),
    ([0, 333, 401, 5], [200, 129, 1, 0], 16, 16, 128, 16, 0),
    ([0, 333, 40, 129], [200, 129, 64, 128], 4, 2, 256, 32, 0),
    ([1000], [300], 12, 4, 128, 128, 0),
    ([63, 64, 65, 127, 128, 129], [1, 2, 63, 64, 65, 127], 2, 1, 128, 64, 0),
    ([31, 32], [33, 96], 16, 1, 128, 16, 0),
    ([7], [50], 15, 3, 256, 64, 0),
    ([0], [515], 8, 8, 256, 128, 0),
    ([0], [700], 4, 4, 128, 64, 1),
    ([0, 2000], [700, 130], 6, 2, 128, 64, 64),
    ([0, 300, 90], [400, 300, 7], 16, 2, 128, 32, 100),
    ([500], [260], 4, 2, 256, 16, 257),
    ([100], [300], 4, 4, 128, 64, 100000),
    ([8193], [3], 8, 2, 128, 64, 0),
    ([20000, 0, 17], [1, 1, 1], 32, 8, 128, 64, 0),
    ([9000], [20], 16, 4, 256, 128, 5000),
    ([i % 7 * 3 for i in range(256)], [20 + i % 3 for i in range(256)], 16, 1, 128, 16, 0),  # 768 row tiles: more than a CTA has threads
    ([0, 5], [10500, 10400], 4, 1, 128, 128, 200),  # the same of two sequences
]


@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(epq_lib, shape):
    c = Case(epq_lib, *shape)
    out = c.check()
    assert epq_lib.epq_device_error() == 0
    assert torch.equal(out, c.run()), "not reproducible"


@pytest.mark.parametrize("D", [128, 256])
def test_long(epq_lib, D):
    c = Case(epq_lib, [4000], [1100], 8, 2, D, 64)
    c.check()
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("spread", [0.0, 0.01, 30.0, 300.0])
def test_spread(epq_lib, spread):
    """Equal weights, nearly equal ones, and one position that takes all."""
    Case(epq_lib, [200, 0], [140, 90], 8, 2, 128, 64, spread=spread, seed=3).check()


@pytest.mark.parametrize("qmul, kmul, vmul", [(1e-20, 1e-3, 1e-4), (1e20, 1e3, 1e5), (1e-30, 1e4, 1.0), (1.0, 1e-5, 4e6), (1.0, 1e-5, 1e6), (1e15, 1e-4, 1e-5)])
def test_scales(epq_lib, qmul, kmul, vmul):
    """Queries, keys and values far from 1, factors that are subnormal halves among them (values above 127 * 65504 = 8.3e6
    have a factor of infinity: with vmul 4e6 that is what most positions have, and NaN what most tokens get)."""
    Case(epq_lib, [150], [100], 8, 2, 128, 64, qmul=qmul, kmul=kmul, vmul=vmul, seed=5).check()


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("what", ["blocks", "positions", "both"])
def test_unequal_rows(epq_lib, what, D):
    """Keys and values whose blocks, or positions, lie 2^30 apart: each output is as exact as its own terms."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T = 300
    e = torch.zeros(T, 1, D // 32, device="cuda")
    if what in ("blocks", "both"):
        e = e + torch.randint(-10, 5, (1, 1, D // 32), generator=g, device="cuda")
    if what in ("positions", "both"):
        e = e + torch.randint(-10, 5, (T, 1, 1), generator=g, device="cuda")
    mul = torch.exp2(e.clamp(-15, 15)).repeat_interleave(32, -1).view(T, 1, D)
    c = Case(epq_lib, [180], [120], 4, 2, D, 64, kmul=1.0 if what == "positions" else mul.clamp(max=4.0), vmul=mul, seed=7)
    c.check()


def test_small_values_behind_large_weights(epq_lib):
    """Codes 0 under every large weight leave outputs that only small weights make."""
    c = Case(epq_lib, [0], [256], 2, 1, 128, 64, seed=9)
    rows = c.rows(0)
    v = rows[:, :, 1, 8:].view(torch.int8)
    v[:, :, :64] = 0
    rows[100:110, :, 1, 8:72] = 1
    k = _values(rows)[:, :, 0].float()
    k[100:110] *= 0.05
    rows[:, :, 0] = _rows(k)
    c.put(0, torch.arange(256, device="cuda"), rows)
    c.check()


def test_not_finite(epq_lib):
    """A position with a factor that is not finite: NaN for the tokens that attend to it, in its head, and nothing else."""
    for plane in (0, 1):
        for bits in (0x7c00, 0x7e00, 0xfc00):  # inf, NaN, -inf
            c = Case(epq_lib, [70, 20], [150, 80], 4, 2, 128, 64, window=90, seed=11)
            clean = c.check()
            page, slot = int(c.c.table[0, 130 // 64]), 130 % 64
            c.c.pool[0, page, 1, plane, slot, 2:4] = torch.tensor([bits & 255, bits >> 8], dtype=torch.uint8)
            got = c.run().view(2, 150, 4, 128)
            want = clean.view(2, 150, 4, 128).clone()
            i = torch.arange(150, device="cuda") + 70
            hit = (i >= 130) & (i < 130 + 90)
            assert torch.isnan(got[0, hit, 2:]).all()
            want[0, hit, 2:] = 0
            got = got.clone()
            got[0, hit, 2:] = 0
            assert torch.equal(got, want)
    assert epq_lib.epq_device_error() == 0


def test_missing_pages(epq_lib):
    """Positions without a page are left out and recorded; a token that sees no other gets 0."""
    c = Case(epq_lib, [100, 0], [100, 70], 4, 2, 128, 16, window=16, seed=13)
    keep = c.c.table.clone()
    rows = [c.rows(s).clone() for s in range(2)]
    c.c.table[0, 7] = -1           # positions 112..127
    c.c.table[1, 0] = c.c.n_pages  # no such page: positions 0..15
    out = c.run()
    assert epq_lib.epq_device_error() == 5
    c.c.table.copy_(keep)
    hide = [torch.arange(112, 128, device="cuda"), torch.arange(0, 16, device="cuda")]
    for s in range(2):
        r = rows[s]
        r[hide[s]] = 0
        c.put(s, torch.arange(len(r), device="cuda"), r)
    c.check(out=out, hidden=hide)
    # token 27 of sequence 0 (position 127) sees 112..127 alone, tokens 0..15 of sequence 1 only what is missing
    assert not out[0, 27].any() and not out[1, :16].any() and out[1, 16:70].any(-1).all()
    # lengths past the table, and below 0, are held to it
    c.c.length.copy_(torch.tensor([2**31 - 1, -5], dtype=torch.int32))
    c.run()
    epq_lib.epq_device_error()


def test_strides_stream_and_workspace(epq_lib):
    """Queries in a wider buffer, sequences side by side, a named stream, a workspace that holds anything, an output that is given."""
    c = Case(epq_lib, [40, 0], [70, 66], 8, 2, 128, 64, seed=15)
    want = c.check()
    wide = torch.full((70, 2, 12 * 128), math.nan, device="cuda")
    q = wide.transpose(0, 1)[..., 128:9 * 128]
    q.copy_(c.q)
    ws = epq_lib.epq_attention_prompt_workspace(c.c, 8, 70)
    ws.fill_(0xff)
    out = torch.full_like(want, 7.0)
    assert c.run(q=q, workspace=ws, out=out) is out and torch.equal(out, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = c.run(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(other, want)


def test_graph(epq_lib):
    """Captured once, replayed with other lengths and queries; two graphs share the workspace."""
    c = Case(epq_lib, [300, 10], [90, 70], 8, 2, 128, 64, seed=17)
    ws = epq_lib.epq_attention_prompt_workspace(c.c, 8, 90)
    out, nt = torch.empty_like(c.q), torch.tensor(c.n_tok, dtype=torch.int32, device="cuda")
    run = lambda o: epq_lib.epq_attention_prompt(c.q, c.c, 0, 8, c.scale, n_tok=nt, out=o, workspace=ws)  # noqa: E731
    run(out)
    torch.cuda.synchronize()
    two = torch.empty_like(out)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, (out, two)):
        with torch.cuda.graph(g):
            run(o)
    for lengths, n_tok in (([300, 10], [90, 70]), ([301, 0], [89, 80]), ([3, 4], [1, 2]), ([0, 0], [0, 0])):
        c.lengths, c.n_tok = lengths, n_tok
        c.c.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        nt.copy_(torch.tensor(n_tok, dtype=torch.int32))
        c.q.normal_(std=2.0)
        for g in graphs:
            g.replay()
        c.check(out=out)
        assert torch.equal(out, two)


def test_layers_and_far_pages(epq_lib):
    """Layers and pages whose bytes lie past 2^32."""
    kv, D, P = 4, 256, 128
    n = (1 << 32) // (kv * 2 * P * 272) + 40
    c = epq_lib.PagedKVCache(2, n // 2, kv, D, 1, 8, P)
    ids = torch.tensor([n // 2 - 1, 0, n // 2 - 7, n // 2 - 2, 5], device="cuda")
    c.table[0, :5] = ids.int()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(600, kv, 2, D, generator=g, device="cuda")
    case = Case(epq_lib, [500], [100], 8, kv, D, P)
    pos = torch.arange(600, device="cuda")
    r = _rows(x)
    case.put(0, pos, r)
    want = case.check()
    c.pool[1, ids[pos // P], :, :, pos % P] = r
    c.length.fill_(500)
    got = epq_lib.epq_attention_prompt(case.q, c, 1, 8, case.scale)
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [5, 64])
def test_agrees_with_the_tree(epq_lib, n):
    """A chain of drafted tokens through epq_attention_tree, and the same rows appended and attended: the same cache, and
    outputs within two bounds of each other."""
    c = Case(epq_lib, [130, 7], [n, n], 8, 2, 128, 64, seed=19)
    x = torch.randn(2, n, 12 * 128, device="cuda")
    q, k, v = x[..., :1024], x[..., 1024:1280], x[..., 1280:]
    tree = epq_lib.epq_attention_tree(q, k, v, c.c, 0, 8, c.scale)
    pool = c.c.pool.clone()
    epq_lib.epq_pages_append(k, v, c.c, 0)
    assert torch.equal(pool, c.c.pool)
    c.q = q.contiguous()
    c.check(out=tree)
    c.check()


def test_prompt_in_chunks(epq_lib):
    """A prompt at once, and in chunks of any length, each appended with its rotation, attended and advanced."""
    tab = epq_lib.RopeTable(128, 512)
    x = torch.randn(1, 400, 12 * 128, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    outs = []
    for chunks in ([400], [1, 64, 65, 200, 70]):
        c = epq_lib.PagedKVCache(1, 8, 2, 128, 1, 8)
        y, at = [], 0
        for n in chunks:
            n_t = torch.tensor([n], dtype=torch.int32, device="cuda")
            assert epq_lib.epq_pages_reserve(c, n_t).tolist() == [0]
            part = x[:, at:at + n]
            q = epq_lib.epq_rope(part[..., :1024], tab, 8, start=c.length)
            epq_lib.epq_pages_append(part[..., 1024:1280], part[..., 1280:], c, 0, rope=tab)
            y.append(epq_lib.epq_attention_prompt(q, c, 0, 8, 128 ** -0.5))
            epq_lib.epq_pages_advance(c, n_t)
            at += n
        assert c.length.tolist() == [400]
        outs.append((torch.cat(y, 1), c.pool.clone(), c.table.clone()))
    assert torch.equal(outs[0][1], outs[1][1]) and torch.equal(outs[0][2], outs[1][2])
    d = (outs[0][0] - outs[1][0]).abs().max().item()
    # weights sum to 1 and scores are a few units: two bounds of a few hundred 2^-24 of values of at most about 5
    assert d <= 2 * 5 * (2 * (32 + 32) * 2.0 ** -24 * 30 + 2 * (32 + 100) * 2.0 ** -24)


def test_bad_pages_and_refusals_leave_no_error(epq_lib):
    c = Case(epq_lib, [10], [20], 4, 2, 128, 16)
    with pytest.raises(epq_lib.EpqError):
        epq_lib.epq_attention_prompt(c.q, c.c, 1, 4, c.scale)
    with pytest.raises(ValueError):
        epq_lib.epq_attention_prompt(c.q.cpu(), c.c, 0, 4, c.scale)
    assert epq_lib.epq_device_error() == 0


@pytest.mark.parametrize("D", [128, 256])
def test_two_at_once(epq_lib, D):
    """Two calls on two streams with workspaces of their own, again and again while the other runs."""
    cs = [Case(epq_lib, [700, 20], [300, 129], 8, 2, D, 64, seed=21), Case(epq_lib, [0, 900], [400, 7], 4, 4, D, 16, window=333, seed=22)]
    want = [c.check() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(6):
        for c, st, o in zip(cs, streams, outs):
            with torch.cuda.stream(st):
                o.append(c.run())
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
    assert epq_lib.epq_device_error() == 0


def test_token_counts_out_of_range(epq_lib):
    """Counts below 0 and above ntok are held to it; no counts are all tokens."""
    c = Case(epq_lib, [10, 20, 30], [40, 40, 40], 4, 2, 128, 16, seed=23)
    want = c.check()
    run = lambda nt: epq_lib.epq_attention_prompt(c.q, c.c, 0, 4, c.scale, n_tok=nt)  # noqa: E731
    assert torch.equal(run(None), want)
    got = run(torch.tensor([2**31 - 1, -3, 41], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[[0, 2]], want[[0, 2]]) and not got[1].any()
    assert epq_lib.epq_device_error() == 0


def test_head_of_256_with_16_queries(epq_lib):
    Case(epq_lib, [40, 333], [30, 77], 16, 1, 256, 32).check()
