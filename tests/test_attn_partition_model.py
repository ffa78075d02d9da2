"""Host model of tree_attn's schedule: shares of the tiles, parts and their slots, and the joining
kernel's blocks.  Every tile of every unit is taken once; a unit is written whole or joined
exactly once from exactly its parts; a block without a unit touches nothing; every slot is
inside the workspace and written by one part."""
import random

import pytest

CTAS = 152
COST = 2   # tiles that a unit counts for beside its own, in front of them


def share(total, ctas, c):
    return total * c // ctas


def walk(units, total, ctas, c):
    """Parts (unit, ta, tb) of CTA c's share; units are (tiles, rows).  Parts without tiles are left out."""
    at, left, u = share(total, ctas, c), share(total, ctas, c + 1) - share(total, ctas, c), 0
    while at >= units[u][0] + COST:
        at -= units[u][0] + COST
        u += 1
    parts = []
    while left > 0:
        end = min(units[u][0] + COST, at + left)
        ta, tb = max(at - COST, 0), max(end - COST, 0)
        if tb > ta:
            parts.append((u, ta, tb))
        left -= end - at
        at, u = 0, u + 1
    return parts


@pytest.mark.parametrize("seed", range(60))
def test_parts_and_joins(seed):
    rng = random.Random(seed)
    kind = rng.choice(["few long", "many short", "mixed"])
    n = {"few long": rng.randint(1, 8), "many short": rng.randint(100, 900), "mixed": rng.randint(1, 300)}[kind]
    units = [({"few long": rng.randint(1, 3000), "many short": rng.randint(1, 3), "mixed": rng.choice([1, 2, 50, 300])}[kind],
              rng.randint(1, 256)) for _ in range(n)]
    total = sum(t + COST for t, _ in units)
    ctas = min(total, CTAS)
    start = [COST]
    for t, _ in units:
        start.append(start[-1] + t + COST)
    taken = [[0] * t for t, _ in units]
    whole, slots, desc = set(), {}, {}
    for c in range(CTAS):
        if c >= ctas:
            desc[c] = (0, None, None, None)                     # rows = 0, the rest left as it was
            continue
        parts = walk(units, total, ctas, c)
        for k, (u, ta, tb) in enumerate(parts):
            for t in range(ta, tb):
                taken[u][t] += 1
            if ta == 0 and tb == units[u][0]:
                whole.add(u)
                continue
            slot = 2 * c + (0 if ta > 0 else 1)
            assert 0 <= slot < 2 * CTAS and slot not in slots
            slots[slot] = u
        desc[c] = (0, None, None, None)
        if parts and parts[0][1] > 0:
            u = parts[0][0]
            begin = start[u]
            first = ((begin + 1) * ctas + total - 1) // total
            last = ((begin + units[u][0]) * ctas + total - 1) // total - 1
            desc[c] = (units[u][1], u, first, last)
    assert all(x == 1 for t in taken for x in t)
    joined, threads, gy = {}, 64, rng.choice([2, 8])            # outputs of a block at a time
    for c in range(1, CTAS):
        rows, u, first, last = desc[c]
        if rows <= 0:
            continue
        assert 1 <= first <= c <= last < ctas
        outputs = rows * 32
        for y in range(gy):
            joined.setdefault(u, []).extend(
                x for t in (0, threads - 1) for x in range(((c - first) * gy + y) * threads + t, outputs, (last - first + 1) * gy * threads))
        parts = {2 * i + (1 if i < first else 0) for i in range(first - 1, last + 1)}
        assert parts == {s for s, v in slots.items() if v == u}
    for u in range(n):
        assert (u in whole) != (u in joined), u
        if u in joined:                                          # the first and the last thread's outputs, each once
            want = [x for x in range(units[u][1] * 32) if x % threads in (0, threads - 1)]
            assert sorted(joined[u]) == want


def test_fast_division():
    """floor(n * ceil(2^s / d) / 2^s) with s = 31 + ceil(log2 d) is n // d for n < 2^31."""
    rng = random.Random(0)
    for d in [1, 2, 3, 5, 7, 16, 24, 255, 256, 1 << 20, (1 << 24) - 1, 1 << 24] + [rng.randint(1, 1 << 24) for _ in range(500)]:
        s = 31
        while 1 << (s - 31) < d:
            s += 1
        mul = ((1 << s) + d - 1) // d
        assert mul < 1 << 32
        top = (1 << 31) - 1
        for n in [0, 1, d - 1, d, d + 1, top, top // d * d, top // d * d - 1] + [rng.randint(0, top) for _ in range(50)]:
            if 0 <= n <= top:
                assert n * mul >> s == n // d
