"""Float64 / whole-number oracle of the paged key/value cache: reservation of slots
by lists, and what a sequence's pages hold. Attention over them is
``oracle.kv4.attend``, which takes rows in order."""
from __future__ import annotations

import numpy as np


def reserve(table, lens, free, n_free, add, page, T):
    """table [B, max_pages], lens [B], free [pages] (the first n_free are the stack), add [B].
    Returns (table, lens, free, n_free, cu, slots, refused): new arrays."""
    table, free = np.array(table), np.array(free)
    B, most = table.shape
    stack = list(free[:n_free])
    for b in range(B):
        if add[b] < 0:
            stack += list(table[b, :-(-lens[b] // page)])
    free[:len(stack)] = stack
    out, slots, cu, refused = list(lens), [], [0], []
    short = False                                    # one before did not find its pages
    for b in range(B):
        n = max(int(add[b]), 0)
        cu.append(cu[-1] + n)
        if add[b] < 0:
            out[b] = 0
            continue
        held = -(-int(lens[b]) // page)
        need = -(-(int(lens[b]) + n) // page) - held
        if lens[b] + n > most * page:
            refused.append(b)
            slots += [-1] * n
            continue
        if need and (short or need > len(stack)):
            short = True
            refused.append(b)
            slots += [-1] * n
            continue
        for j in range(need):
            table[b, held + j] = stack.pop()
        out[b] = lens[b] + n
        slots += [int(table[b, s // page]) * page + s % page for s in range(lens[b], out[b])]
    slots = (slots + [-1] * T)[:T]
    return table, np.array(out), free, len(stack), np.array(cu), np.array(slots), refused


def rows(pool, pages, n, h, page):
    """The first n slots of head h of a sequence with these pages; pool [pages, Hkv, page, D]."""
    return pool[np.asarray(pages[:-(-n // page)], dtype=int), h].reshape(-1, pool.shape[-1])[:n]
