"""The accuracy that epq.h states for epq_attention_prompt, elementwise against 64 bits, in units of 2^-24.

A score: products of two-part operands leave out 8 units (2^-10 of the one times 2^-11 of the other) and round a
query's rest (4); D/16 steps of the tensor core add 16 products each to one sum, 4 units each; the scale, the
exponential's argument and its reference take fewer than 20.  At most 32 + D/4 of scale sum |q||k|, and since most of
these have either sign, some 16 (2^-20) on numbers of either sign.

An output, beside that: a weight's exponential (4, in the sum and in the output: 8), its rest (4), the product of
rests (8), 64 additions of a tile's weights in a row (64), a tile's products with values in at most 8 steps (32), the
quotient (2): 118, whatever T is.  Each tile's sum is a fresh one; what grows with T is its addition to the output and
to the weights' sum, and the factor between two references (its exponential 4, its products 2): 8 for each tile, T D /
2048 in all.  The join of two parts takes no more than the step between two tiles.  At most 128 + T D / 2048 of sum
w|v|, and on numbers of either sign, or equal weights, some 32 (2^-19) at any T.

Floors: a weight is off by up to 2^-39 of its row's largest, an element whose factor is below 2^-21 of the largest
among its tile's (128 positions, 64 for heads of 256; of a value in its 32 columns, of a key in all) by up to 2^-32 of
its code times that largest factor."""
import math

import pytest
import torch
from test_gpu_prompt_attention import Case, _rows, _values

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24


def _floors(rows, D):
    """What the elements of rows [T, kv, 2, row] may be off by: [T, kv, 2, D]."""
    T, kv = rows.shape[:2]
    P = 128 if D == 128 else 64
    f = rows[..., : D // 16].contiguous().view(torch.float16).double()
    codes = rows[..., D // 16:].contiguous().view(torch.int8).double().abs()
    pad = torch.zeros(-T % P, *f.shape[1:], dtype=f.dtype, device=f.device)
    top = torch.cat([f, pad]).view(-1, P, kv, 2, D // 32).amax(1)
    top[:, :, 0] = top[:, :, 0].amax(-1, keepdim=True)
    top = top.repeat_interleave(P, 0)[:T]
    return codes * torch.where(f < 2.0 ** -21 * top, 2.0 ** -32 * top, 0.0).repeat_interleave(32, -1)


def _worst(c, score, output, out=None):
    """The largest error over its bound: `score` units of scale sum |q||k|, `output` units of sum w|v|."""
    out = c.run() if out is None else out
    D, G, worst = c.D, c.heads // c.kv, 0.0
    got = out.view(len(c.lengths), c.ntok, c.heads, D).double()
    for s, (n, t) in enumerate(zip(c.lengths, c.n_tok)):
        see = n + torch.arange(t, device="cuda")[:, None] >= torch.arange(n + t, device="cuda")
        rows = c.rows(s)
        x, fl = _values(rows), _floors(rows, D)
        for h in range(c.kv):
            K, V, fk, fv = x[:, h, 0], x[:, h, 1], fl[:, h, 0], fl[:, h, 1]
            q = c.q[s, :t].view(t, c.heads, D)[:, h * G:(h + 1) * G].double()
            w = torch.softmax((q @ K.T * c.scale).masked_fill(~see[:, None], -math.inf), -1)
            mag = lambda k: (q.abs() @ k.T * c.scale).masked_fill(~see[:, None], 0.0).amax(-1, keepdim=True)  # noqa: E731
            grow = torch.expm1(2 * (score * UNIT * mag(K.abs()) + mag(fk)))
            bound = (w @ V.abs()) * (grow + output * UNIT) + (w @ fv) * (1 + grow) + 2.0 ** -39 * V.abs().sum(0) + 1e-30
            off = (got[s, :t, h * G:(h + 1) * G] - w @ V).abs() / bound
            assert not torch.isnan(off).any()
            worst = max(worst, off.max().item())
    return worst


CASES = [  # lengths, n_tok
    ([0], [130]), ([5000], [100]), ([19980], [20]),
]


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("spread", [0.0, 0.5, 2.0])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_stated_accuracy(epq_lib, case, positive, spread, D):
    """2^-20 of a score's terms, 2^-19 of an output's, over 130 positions and over 20000; positive: values, and keys and
    queries, of one sign, whose sums only grow."""
    c = Case(epq_lib, *case, 4, 2, D, 64, spread=spread, seed=27)
    if positive:
        c.q.abs_()
        rows = c.rows(0)
        c.put(0, torch.arange(len(rows), device="cuda"), _rows(_values(rows).float().abs()))
        c.scale /= 4.0
    T = case[0][0] + case[1][0]
    out = c.run()
    assert _worst(c, 32 + D / 4, 128 + T * D / 2048, out) <= 1
    assert _worst(c, 16, 32, out) <= 1


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("apart", [20, 24, 27, 30])
def test_values_apart(epq_lib, apart, D):
    """A tile whose last value row has factors 2^apart times the others': outputs of the tokens before it are made of the
    others alone."""
    T = 300
    mul = torch.full((T, 1, 1), 2.0 ** -13, device="cuda")
    mul[63::64] = 2.0 ** (apart - 13)
    c = Case(epq_lib, [0], [T], 4, 2, D, 64, kmul=torch.ones(1, 1, 1, device="cuda"), vmul=mul, seed=29, spread=1.0)
    f = c.rows(0)[:, :, 1, : D // 16].contiguous().view(torch.float16).float()
    assert f[63].min() >= 2.0 ** (apart - 3) * f[:63].max() and f[:63].max() > 0
    assert _worst(c, 32 + D / 4, 128 + T * D / 2048) <= 1


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("apart", [20, 24, 27, 30])
def test_keys_apart(epq_lib, apart, D):
    """Keys whose first 32 columns have factors 2^apart times the others', under queries that are 0 there: scores that
    the others make alone."""
    mul = torch.full((1, 1, D // 32), 2.0 ** -13, device="cuda")
    mul[..., 0] = 2.0 ** (apart - 13)
    c = Case(epq_lib, [100], [150], 4, 2, D, 64, kmul=mul.repeat_interleave(32, -1), seed=31, spread=1.0)
    c.q.view(1, 150, 4, D)[..., :32] = 0.0
    c.scale *= 2.0 ** 13
    f = c.rows(0)[:, :, 0, : D // 16].contiguous().view(torch.float16).float()
    assert f[..., 0].min() >= 2.0 ** (apart - 3) * f[..., 1:].max() and f[..., 1:].max() > 0
    assert _worst(c, 32 + D / 4, 128 + 250 * D / 2048) <= 1
