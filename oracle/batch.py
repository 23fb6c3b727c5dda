"""Plain oracle of a paged batch's step: pages and places for its tokens, norms
and rotary positions, and the rows that a shared prefix stands for.  Test
infrastructure only; one function per step, in float64 and Python integers,
nothing shared with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def plan(table, counts, start, first, shared, held, ring, span, page, n_slots, n_pages):
    """What a plan leaves: dict of table, ring, span, held, granted, lens, seen (None
    where the sequence is left as it is), starts, slots, and the errors met."""
    table, ring = [list(map(int, row)) for row in table], [int(x) for x in ring]
    S, cap, rows = len(counts), len(ring), len(table[0]) * page
    head, avail = (int(x) for x in span)
    errors = set()
    if not (0 <= head < cap and 0 <= avail <= cap):
        errors.add("count")
        head = avail = 0
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + max(0, int(c)))
    wanted = taken = 0
    handed = []
    out = dict(held=[], granted=[], lens=[], seen=[])
    served = []
    for s in range(S):
        n, c, f, h, sh = int(start[s]), int(counts[s]), int(first[s]), int(held[s]), int(shared[s])
        fine = (n >= 0 and c >= 0 and f >= 0 and 0 <= sh <= h <= len(table[s]) and n + c <= rows
                and f + c <= 2 ** 31 - 1 and (c == 0 or starts[s + 1] <= n_slots))
        if not fine:
            errors.add("count")
            for key, value in (("held", h), ("granted", 0), ("lens", None), ("seen", None)):
                out[key].append(value)
            served.append(False)
            continue
        need = max(sh, -(-(n + c) // page))
        ok = True
        if need > h:
            wanted += need - h
            ok = wanted <= avail
            if ok:
                for i in range(h, need):
                    table[s][i] = ring[(head + taken) % cap]
                    taken += 1
        else:
            handed += table[s][need:h]
        got = c if ok else 0
        for key, value in (("held", need if ok else h), ("granted", got), ("lens", n + got), ("seen", f + got)):
            out[key].append(value)
        served.append(ok)
    if avail + len(handed) > cap:
        errors.add("count")
        handed = handed[:cap - avail]
    for i, p in enumerate(handed):
        ring[(head + avail + i) % cap] = p
    slots = [[-1] * 4 for _ in range(n_slots)]
    for s in range(S):
        if not served[s]:
            continue
        for j in range(out["granted"][s]):
            row = int(start[s]) + j
            p = table[s][row // page]
            if 0 <= p < n_pages:
                slots[starts[s] + j] = [p * page + row % page, s, row, int(first[s]) + j]
            else:
                errors.add("index")
    return dict(out, table=table, ring=ring, span=[(head + taken) % cap, avail - taken + len(handed)],
                starts=[min(x, n_slots) for x in starts], slots=slots, errors=errors)


def rotary(x, position, turns, rot, interleaved, weight=None, eps=0.0, amplitude=1.0):
    """One row x [d] normed and rotated; turns: integers, 2^64 to a turn."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / math.sqrt(float(np.mean(y * y)) + eps) * np.asarray(weight, dtype=np.float64)
    got = y.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = 2 * math.pi * (int(position) * int(turns[i]) % 2 ** 64) / 2 ** 64
        got[a] = amplitude * (y[a] * math.cos(t) - y[b] * math.sin(t))
        got[b] = amplitude * (y[b] * math.cos(t) + y[a] * math.sin(t))
    return got


def groups(starts, prefix, lens, seqs, rows):
    """[(first, end, shared rows)] as the shared attention takes its arguments."""
    got, top = [], 0
    clean = []
    for x in starts:
        top = max(top, min(max(int(x), 0), seqs))
        clean.append(top)
    for i, p in enumerate(prefix):
        a, b = clean[i], clean[i + 1]
        shared = 0
        if b - a > 1:
            shared = min(max(int(p), 0), min(max(int(lens[a]), 0), rows)) // 16 * 16
        got.append((a, b, shared))
    return got
