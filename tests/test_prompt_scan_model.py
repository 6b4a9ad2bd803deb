"""CPU model of how the prompt attention's two scanning warps meet for each tile (host logic; no GPU).

Each warp, for tile g: bounded waits (for the item, for the tile's place), any of which may give up; its note in slot
g % 2; the barrier of both; the partner's note.  A warp that gives up writes "gone" as its note of tile g and arrives
at the barrier without waiting; one that reads "gone" leaves.  Every order of the two warps' steps is walked through:
each must end with both warps gone, and a note must be the one of the tile, and be read before it is written over."""
import os

import pytest

TILES = 5
WAIT, NOTE, SYNC, READ, FAIL, LAST, GONE = range(7)
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_experts_gb300", "csrc",
                      "attention_prompt.cu")


def _write(me, other, what):
    step, g, notes, arrived = me
    assert other[0] != READ or other[1] % 2 != g % 2 or other[1] == g, "a note is written while it is read"
    assert other[0] != SYNC or other[1] >= g - 1, "a note is written before it is read"
    return tuple((what, g) if k == g % 2 else n for k, n in enumerate(notes))


def _steps(me, other, leave):
    """What a warp's next step makes of it: (step, tile, notes, arrivals).  leave: how one that gave up goes."""
    step, g, notes, arrived = me
    if step == WAIT:
        return [(FAIL, g, notes, arrived), (GONE if g == TILES else NOTE, g, notes, arrived)]
    if step == NOTE:
        return [(SYNC, g, _write(me, other, "note"), arrived + 1)]
    if step == SYNC:  # both have arrived as often
        return [(READ, g, notes, arrived)] if other[3] >= arrived else []
    if step == READ:
        what, tile = other[2][g % 2]
        if what == "gone" and leave == "told":
            assert tile == g
            return [(GONE, g, notes, arrived)]
        assert tile == g or leave != "told", "another tile's note"
        return [(WAIT, g + 1, notes, arrived)]
    if step == FAIL:
        if leave == "told":
            return [(LAST, g, _write(me, other, "gone"), arrived)]
        return [(GONE, g, notes, arrived + (leave == "arrives"))]
    if step == LAST:
        return [(GONE, g, notes, arrived + 1)]
    return []


def _stuck(leave):
    """States in which a warp is not gone and nothing can happen."""
    none = (("", -1), ("", -1))
    start = ((WAIT, 0, none, 0),) * 2
    seen, todo, stuck = {start}, [start], []
    while todo:
        s = todo.pop()
        nxt = [(a, s[1]) for a in _steps(s[0], s[1], leave)] + [(s[0], b) for b in _steps(s[1], s[0], leave)]
        if not nxt and any(w[0] != GONE for w in s):
            stuck.append(s)
        for t in nxt:
            if t not in seen:
                seen.add(t)
                todo.append(t)
    return stuck


def test_every_order_ends():
    assert not _stuck("told")


@pytest.mark.parametrize("leave", ["silent", "arrives"])
def test_the_model_sees_a_partner_that_waits(leave):
    """A warp that leaves without a word, or with one arrival alone, leaves the other in the barrier of some tile."""
    assert any(SYNC in (s[0][0], s[1][0]) for s in _stuck(leave))


def test_the_kernel_has_this_barrier_alone():
    """The roles' only barrier without a limit is the one of the scanning warps; all ways out of their loops but the end
    and "gone" go past the arrival."""
    with open(SOURCE, encoding="utf-8") as f:
        text = f.read()
    roles = text[text.index("void copies_role("):text.index("prompt_kernel(const __grid_constant__")]
    assert roles.count("named_sync(") == 1 and roles.count("bar.") == 1 and "__syncthreads" not in roles
    scan = roles[roles.index("void scan_role("):roles.index("struct Piece")]
    assert scan.count("return;") == 2 and "if (it.tiles == 0) return;" in scan and "if (other[5] == kGone) return;" in scan
    tail = scan[scan.index("\ngone:"):]
    assert tail.index("= kGone;") < tail.index("bar.arrive 1, 64;") and "return" not in tail[:tail.index("bar.arrive")]
