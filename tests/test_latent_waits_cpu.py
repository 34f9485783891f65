"""The waits of the absorbed form's kernel, without a GPU: no warp waits without a limit for one that has given up."""
import itertools
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "rotation_quantized_kv_rq_gb300", "csrc", "rq_latent_attention.cu")


def source():
    with open(SOURCE) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def warp(outcomes, tiles, carries):
    """One of the four softmax warps that meet once a tile.  outcomes: whether its waits of a tile before the meeting, and behind it,
    end in time.  Yields what it brings to a meeting and is sent whether it ends it.  carries: a warp whose wait ran out goes to the next
    meeting and says so; otherwise it leaves."""
    ok = True
    for t in range(tiles):
        before, behind = outcomes[t]
        if not (ok and before):
            if carries:
                yield False
            return
        if not (yield True):
            return
        if not behind:
            if not carries:
                return
            ok = False


def all_end(outcomes, tiles, carries):
    """Four warps: a meeting takes place when all four are there; False where some are and others never will be."""
    warps = [warp(o, tiles, carries) for o in outcomes]
    here = [next(w, None) for w in warps]
    while any(h is not None for h in here):
        if any(h is None for h in here):
            return False
        agreed = all(here) if carries else True
        here = [step(w, agreed) for w in warps]
    return True


def step(w, value):
    try:
        return w.send(value)
    except StopIteration:
        return None


@pytest.mark.parametrize("tiles", [1, 2])
def test_four_warps_leave_together(tiles):
    """Whatever waits run out, every warp ends; and not where the warps leave one by one."""
    every = list(itertools.product(itertools.product((True, False), repeat=2), repeat=tiles))
    cases = list(itertools.product(every, repeat=4))
    assert all(all_end(c, tiles, True) for c in cases)
    assert not all(all_end(c, tiles, False) for c in cases)


def test_the_kernel_meets_that_way():
    """The softmax's loop has one meeting a tile of part of a block's warps; it carries their state, and no warp leaves the loop
    but through it (rows past the last one, whose four warps take another way together, aside)."""
    text = source()
    body = text[text.index("auto o_is_done"):text.index("} else if (warp == kMmaWarp)")]
    body = body[body.index("for (int t = 0; t < n; ++t)"):]
    idle = re.search(r"if \(idle\) \{.*?continue;\s*\}", body, re.S)
    rest = body[:idle.start()] + body[idle.end():]
    assert "bar.red.and.pred" in text and not re.search(r"bar\.sync %0", text)
    assert len(re.findall(r"rows_agree\(", rest)) == 2
    assert re.search(r"if \(!ok\) \{\s*rows_agree\(quad & 1, false\);\s*break;\s*\}", rest)
    assert re.search(r"if \(!\(ok = rows_agree\(quad & 1, true\)\)\) break;", rest)
    assert len(re.findall(r"\bbreak;", rest)) == 2 and "return" not in rest
    assert len(re.findall(r"o_is_done\([^)]*\)\)\) continue;", rest)) == 2
