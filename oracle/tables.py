"""Page tables from request lengths, by a stack popped and pushed one page at a time.

Test infrastructure only (see ``oracle/__init__.py``).  The paged cache and its table are the pages'
("Integrate FP32 v37 prefill and exact E4M3 bridge", Implementation); who hands pages out is not
theirs.
"""

import numpy as np


def extend(table, lens, new, stack, page):
    """New tokens for every sequence: pages from the end of `stack` (a list, popped), in the order of
    the sequences; one that needs more than the stack holds, or that needs any behind such a one,
    gets none.  Returns (table, lens, stack, [(positions, slots) per sequence], refused)."""
    table, lens, stack = table.copy(), list(lens), list(stack)
    tokens, refused, short = [], [], False
    for b, m in enumerate(new):
        n = lens[b]
        have = -(-n // page)
        need = -(-(n + m) // page) - have
        short = short or need > len(stack)
        if short and need:
            refused.append(b)
            tokens.append(([-1] * m, [-1] * m))
            continue
        for j in range(need):
            table[b, have + j] = stack.pop()
        lens[b] = n + m
        where = list(range(n, n + m))
        tokens.append((where, [int(table[b, t // page]) * page + t % page for t in where]))
    return table, lens, stack, tokens, refused


def packed(tokens, size):
    """(positions, slots, starts) of the sequences' tokens end to end, -1 up to `size`."""
    starts = np.cumsum([0] + [len(p) for p, _ in tokens])
    out = np.full((2, size), -1, dtype=np.int32)
    for (p, s), at in zip(tokens, starts):
        n = max(0, min(len(p), size - at))
        out[0, at:at + n], out[1, at:at + n] = p[:n], s[:n]
    return out[0], out[1], starts.astype(np.int32)


def rows(tokens, width):
    """(positions, slots) [B][width], a row per sequence, -1 past its tokens."""
    out = np.full((2, len(tokens), width), -1, dtype=np.int32)
    for b, (p, s) in enumerate(tokens):
        out[0, b, :len(p)], out[1, b, :len(s)] = p, s
    return out[0], out[1]


def release(table, lens, keep, stack, page, capacity):
    """The stack (a list) after every sequence's pages behind those of its first keep[b] tokens were
    pushed; from the first sequence on whose pages do not fit, none."""
    stack, short = list(stack), False
    for b, n in enumerate(lens):
        gone = [int(p) for p in table[b, -(-keep[b] // page):-(-n // page)]]
        short = short or len(stack) + len(gone) > capacity
        if not short or not gone:
            stack += gone
    return stack
