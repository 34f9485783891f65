"""The absorbed form's kernel after a wait that ran out, without a GPU: no warp waits without a limit for one that has given up,
and the join finds a note for every unit."""
import itertools
import os
import random
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


OPEN = 3  # what a unit counts for beside its tiles


def cut(tiles, pairs):
    """The ranges of units of so many tiles, cut evenly: parts, and the first of each in tiles (and a unit's opening)."""
    total = sum(t + OPEN for t in tiles)
    parts = min(pairs, total)
    each, more = divmod(total, parts)
    return [c * each + min(c, more) for c in range(parts + 1)]


def notes(tiles, starts):
    """Each unit's note, from the ranges alone: its first range, its parts (0: whole), whether it is that range's last unit of two."""
    holds = lambda x: max(c for c in range(len(starts) - 1) if starts[c] <= x)  # noqa: E731
    at, out = 0, []
    for t in tiles:
        first, last = holds(at + OPEN), holds(at + OPEN + t - 1)
        out.append((first, last - first + 1 if last > first else 0, starts[first] < at))
        at += OPEN + t
    return out


def test_notes_name_the_parts_that_the_ranges_leave():
    rng = random.Random(3)
    for _ in range(300):
        tiles = [rng.choice((1, 1, 2, 5, 40, 300)) for _ in range(rng.randint(1, 40))]
        pairs = rng.choice((1, 2, 7, 76))
        starts = cut(tiles, pairs)
        found = notes(tiles, starts)
        at = 0
        for t, (first, parts, last_of_two) in zip(tiles, found):
            own = [c for c in range(len(starts) - 1) if max(starts[c], at + OPEN) < min(starts[c + 1], at + OPEN + t)]
            assert own == list(range(first, first + max(1, parts))) and parts != 1 and first + parts <= pairs
            # its first range's slot 1, where that range begins with another unit (slot 0)
            assert last_of_two == (starts[first] < at)
            at += OPEN + t


def test_notes_are_written_before_any_wait():
    """Every unit's, before the loop over fragments: a range that ends early leaves no unit without one."""
    text = source()
    written = [m.start() for m in re.finditer(r"\binfo\[", text[:text.index("latent_join_kernel")])]
    kernel = text.index("latent_kernel(const __grid_constant__")
    fragments = text.index("bool first_frag = true;", kernel)
    first_wait = min(text.index(w, kernel) for w in ("barrier.cluster.wait", "warp_wait(", "soft_sync()"))
    assert len(written) == 1 and kernel < written[0] < fragments < first_wait
