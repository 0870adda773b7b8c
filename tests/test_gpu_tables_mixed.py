"""kv_paged_extend over random batches that mix what the other tests look at one at a time -- rejected lengths,
too few pages, more tokens than entries, rows and packed tokens, in place and not -- against the call's
definition, a sequence and a token at a time."""

import numpy as np
import pytest

from tests.test_gpu_tables import t

pytestmark = pytest.mark.gpu


def defined(gb, table, lens, new, stack, page, rows, tokens):
    """(table, lengths, count, starts, positions, slots, flags); `rows` 0: packed, with `tokens` entries."""
    width, F = table.shape[1], len(stack)
    cap, flags, table, out = width * page, 0, table.copy(), list(lens)
    sound = [0 <= n <= cap and 0 <= m <= cap - n and not (rows and m > rows) for n, m in zip(lens, new)]
    wild = [not s and (m < 0 or m > max(tokens, cap)) for s, m in zip(sound, new)]
    places = [m if s or not (rows or x) else 0 for s, m, x in zip(sound, new, wild)]
    if not rows and sum(places) > tokens and any(wild):
        places = [p if s else 0 for s, p in zip(sound, places)]
    starts = np.cumsum([0] + places)
    if not all(sound) or (not rows and starts[-1] > tokens):
        flags |= gb.DEV_BAD_LENGTH
    pos, slots = np.full((2, tokens), -1)
    asked = gone = 0        # pages that the sequences so far need; that are off the stack
    for b, (n, m) in enumerate(zip(lens, new)):
        if not sound[b]:
            continue
        first, held = asked, -(-n // page)
        asked += -(-(n + m) // page) - held
        if asked > F and asked > first:
            flags |= gb.DEV_NO_PAGES
            continue
        for j in range(asked - first):
            table[b, held + j] = stack[F - 1 - first - j]
        have = m if rows else max(0, min(m, int(tokens - starts[b])))
        if -(-(n + have) // page) > held:
            gone = first + -(-(n + have) // page) - held
        out[b] = n + have
        at = (b * rows if rows else starts[b]) + np.arange(have)
        pos[at] = n + np.arange(have)
        slots[at] = table[b, pos[at] // page] * page + pos[at] % page
    return table, out, F - gone, starts, pos, slots, flags


def batch(rng):
    page, width = int(rng.choice([16, 32, 64])), int(rng.integers(1, 12))
    cap, B, top = page * width, int(rng.choice([1, 2, 3, 7, 33, 200, 700])), int(rng.choice([2, 20, page * width]))
    lens = [int(x) for x in rng.integers(0, cap + 1, B)]
    new = [int(min(rng.integers(0, top + 1), cap - n)) for n in lens]
    if rng.random() < 0.6:
        for b in rng.integers(0, B, max(1, B // 5)):
            kind = rng.integers(0, 6)
            if kind == 0:
                new[b] = int(cap - lens[b] + rng.integers(1, 9))
            elif kind == 1:
                lens[b] = -int(rng.integers(1, 9))
            elif kind == 2:
                lens[b] = cap + int(rng.integers(1, 9))
            elif kind == 3:
                lens[b], new[b] = cap, max(1, min(new[b], cap))
            elif rng.random() < 0.3:
                new[b] = (-3, 2 ** 31 - 1)[kind - 4]
    held = [-(-n // page) if 0 <= n <= cap else 0 for n in lens]
    need = sum(-(-min(n + max(m, 0), cap) // page) - h for n, m, h in zip(lens, new, held) if 0 <= n <= cap)
    order = rng.permutation(max(1, sum(held) + (need + 3 if rng.random() < 0.6 else int(rng.integers(0, need + 4)))))
    table, at = np.full((B, width), -1, dtype=np.int32), 0
    for b, c in enumerate(held):
        table[b, :c] = order[at:at + c]
        at += c
    total = sum(m for m in new if 0 <= m <= cap + 20)
    rows = int(rng.integers(1, top + 2)) if rng.random() < 0.3 else 0
    some = total + int(rng.integers(0, 5)) if rng.random() < 0.5 else int(rng.random() * (total + 3))
    return table, lens, new, order[at:].tolist(), page, rows, B * rows if rows else max(1, some)


@pytest.mark.parametrize("seed", range(4))
def test_random_batches(gb, seed):
    rng = np.random.default_rng(seed)
    for i in range(100):
        table, lens, new, stack, page, rows, tokens = batch(rng)
        rt, rl, count, starts, pos, slots, flags = defined(gb, table, lens, new, stack, page, rows, tokens)
        cap, P = table.shape[1] * page, max(1, int((table >= 0).sum()) + len(stack))
        everything = sorted(table[table >= 0].tolist() + stack)
        for in_place in (False, True):
            gt, gl, gc = t(table), t(lens), t([len(stack)])
            kw = dict(row_tokens=rows) if rows else dict(max_tokens=tokens)
            if in_place:
                kw.update(kv_lens_out=gl, free_count_out=gc)
            out = gb.kv_paged_extend(gt, gl, t(new), t(stack + [-7]), gc, page, P, **kw)
            assert gb.device_status() == flags, i
            assert out[0].tolist() == rl and out[1].item() == count and out[2].tolist() == starts.tolist(), i
            assert np.array_equal(out[3].flatten().cpu().numpy(), pos), i
            assert np.array_equal(out[4].flatten().cpu().numpy(), slots), i
            got = gt.cpu().numpy()
            held = [(b, -(-n // page)) for b, n in enumerate(rl) if 0 <= n <= cap]
            assert all(np.array_equal(got[b, :n], rt[b, :n]) for b, n in held), i
            mine = [p for b, n in held for p in got[b, :n].tolist()]
            assert sorted(mine + stack[:count]) == everything, i      # every page once
