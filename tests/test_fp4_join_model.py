"""Model of how the draining warps of the streaming kernel (exq_fp4_stream.cuh) hear from one of them whether a tile's parts are all
there: after a part is written (`last`), and before the sums of the CTA's last tile are taken (`there`). Every interleaving of two
warps is tried; all of them must read what was written for the tile they are at, or they part ways at the next barrier."""
from __future__ import annotations

import pytest

BAR = "bar"


def _programs(word):
    """Steps of the warp that decides and of another, for a tile that began in an earlier CTA, then the CTA's last one."""
    leader = [BAR, ("write", "last", 1), BAR, ("read", "last", 1), ("write", word, 2), BAR, ("read", word, 2)]
    other = [BAR, BAR, ("read", "last", 1), BAR, ("read", word, 2)]
    return leader, other


def _wrong_reads(word):
    programs, wrong, seen = _programs(word), set(), set()

    def run(at, memory):
        if (at, memory) in seen:
            return
        seen.add((at, memory))
        heads = [p[i] if i < len(p) else None for p, i in zip(programs, at)]
        if all(h == BAR for h in heads):
            run(tuple(i + 1 for i in at), memory)
        for w, h in enumerate(heads):
            if h is None or h == BAR:
                continue
            kind, name, value = h
            now = dict(memory)
            if kind == "write":
                now[name] = value
            elif now[name] != value:
                wrong.add((w, name, now[name]))
            run(tuple(i + (j == w) for j, i in enumerate(at)), tuple(sorted(now.items())))

    run((0, 0), (("last", 0), ("there", 0)))
    assert (tuple(len(p) for p in programs)) in {at for at, _ in seen}  # every way ends
    return wrong


@pytest.mark.parametrize("word,sound", [("last", False), ("there", True)])
def test_the_last_tile_has_a_word_of_its_own(word, sound):
    assert (not _wrong_reads(word)) == sound
