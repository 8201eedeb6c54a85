"""CPU model of the barriers between the scores, the softmax and the values of the attention kernel of many rows (host
logic, no GPU).

S of tile g completes phase g // 4 of barrier g % 4 of s_full; P V of it the same of pv_done, which takes an arrival of
each of the two M tiles; the scores of tile g are issued when P V of tile g - 2 is over. The softmax of an M tile waits for
s_full and arrives on w_full of the tile's buffer, the issuer of its values waits for w_full. A unit of at most 128 rows
leaves the second M tile without rows: its softmax and its issuer only keep the phases whole. Every wait is a parity wait
on four barriers, so a role that is four tiles late waits for a phase that has gone by.

The model runs the roles under random interleavings, some of them slow, and checks that no wait meets a barrier which is
more than one phase past the awaited one (or one short of it). Where the softmax without rows only watches s_full, nothing
waits for it and the model finds it four tiles late. In the chain (it arrives on w_full, and its issuer waits for that),
the model finds none.
"""
from __future__ import annotations

import random

SCORES, SOFTMAX, VALUES = "scores", "softmax", "values"


def _run(units, chained, rng):
    """units: (tiles, the second M tile has rows). Returns "ok", "missed" or "deadlock"."""
    tiles = [(active, j == n - 1) for n, active in units for j in range(n)]
    T = len(tiles)
    s_full, pv_done, pv_arrived = [0] * 4, [0] * 4, [0] * 4   # completed phases; arrivals of pv_done's phase
    w_full = [[0, 0], [0, 0]]                                 # [M tile][buffer], completed phases
    at = {SCORES: 0, (SOFTMAX, 0): 0, (SOFTMAX, 1): 0, (VALUES, 0): 0, (VALUES, 1): 0}
    stage = {(SOFTMAX, 0): 0, (SOFTMAX, 1): 0}                # 0: the tile, 1: the unit's last P V, 2: the epilogue
    slow = {k: rng.choice([1, 1, 4, 30]) for k in at}         # a role's steps are that many times rarer

    def missed(completed, phase):
        return completed > phase + 1

    for _ in range(100000):
        if all(v == T for v in at.values()):
            return "ok"
        acts = []
        g = at[SCORES]
        if g < T and (g < 2 or pv_done[(g - 2) & 3] > (g - 2) >> 2):
            acts.append((SCORES, None))
        for s in (0, 1):
            g = at[(SOFTMAX, s)]
            if g < T:
                active, last = tiles[g][0] or s == 0, tiles[g][1]
                if stage[(SOFTMAX, s)] == 0:
                    if missed(s_full[g & 3], g >> 2):
                        return "missed"
                    if s_full[g & 3] > g >> 2:
                        acts.append((SOFTMAX, s))
                elif stage[(SOFTMAX, s)] == 1:
                    if missed(pv_done[g & 3], g >> 2):
                        return "missed"
                    if pv_done[g & 3] > g >> 2:
                        acts.append((SOFTMAX, s))
                else:
                    acts.append((SOFTMAX, s))
            g = at[(VALUES, s)]
            if g < T:
                active = tiles[g][0] or s == 0
                if active or chained:
                    done, phase = w_full[s][g & 1], _weights_before(tiles, g, s, chained)
                else:
                    done, phase = s_full[g & 3], g >> 2
                if missed(done, phase):
                    return "missed"
                if done > phase:
                    acts.append((VALUES, s))
        if not acts:
            return "deadlock"
        kind, s = rng.choices(acts, [1 / slow[a if a[0] != SCORES else SCORES] for a in acts])[0]
        if kind == SCORES:
            s_full[at[SCORES] & 3] += 1
            at[SCORES] += 1
        elif kind == SOFTMAX:
            g = at[(SOFTMAX, s)]
            active, last = tiles[g][0] or s == 0, tiles[g][1]
            step = stage[(SOFTMAX, s)]
            if step == 0 and (active or chained):
                w_full[s][g & 1] += 1
            if active and last and step < 2:
                stage[(SOFTMAX, s)] = step + 1
            else:
                stage[(SOFTMAX, s)] = 0
                at[(SOFTMAX, s)] += 1
        else:
            g = at[(VALUES, s)]
            pv_arrived[g & 3] += 1
            if pv_arrived[g & 3] == 2:
                pv_arrived[g & 3] = 0
                pv_done[g & 3] += 1
            at[(VALUES, s)] += 1
    return "deadlock"


def _weights_before(tiles, g, s, chained):
    """Phases of w_full of tile g's buffer that come before tile g's."""
    return sum(1 for i in range(g & 1, g, 2) if chained or tiles[i][0] or s == 0)


def _outcomes(chained):
    rng = random.Random(7)
    out = []
    for _ in range(400):
        units = [(rng.randint(1, 12), rng.random() < 0.4) for _ in range(rng.randint(1, 6))]
        out.append(_run(units, chained, rng))
    return out


def test_softmax_without_rows_is_in_the_chain():
    assert set(_outcomes(True)) == {"ok"}


def test_model_finds_the_missing_back_pressure():
    got = _outcomes(False)
    assert "missed" in got and "ok" in got
