"""Page tables where a batch brings more tokens than there are entries for their slots (kv_paged_extend):
lengths and pages advance by the tokens that have slots alone."""

import numpy as np
import pytest

from oracle import tables as OT
from tests.test_gpu_tables import make, t

pytestmark = pytest.mark.gpu


def held(lens, page):
    return [-(-n // page) for n in lens]


def entries(new, tokens):
    """Of each sequence's new tokens, those among the first `tokens` end to end."""
    return [max(0, min(m, tokens - at)) for m, at in zip(new, np.cumsum([0] + list(new)))]


def run_cut(gb, lens, new, page, width, spare, tokens, in_place, seed=1):
    table, stack, pages, P = make(lens, page, spare, width, seed)
    kept = entries(new, tokens)
    rt, rl, rs, _, refused = OT.extend(table, lens, kept, stack, page)
    _, _, _, toks, short = OT.extend(table, lens, new, stack, page)
    assert not refused and not short
    gt, gl, gc = t(table), t(lens), t([len(stack)])
    kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
    out = gb.kv_paged_extend(gt, gl, t(new), t(pages), gc, page, P, max_tokens=tokens, **kw)
    assert gb.device_status() == (gb.DEV_BAD_LENGTH if sum(new) > tokens else 0)
    assert out[0].tolist() == rl and out[1].item() == len(rs)
    got = gt.cpu().numpy()
    for b, n in enumerate(held(rl, page)):
        assert np.array_equal(got[b, :n], rt[b, :n]), b
    pos, slots, starts = OT.packed(toks, tokens)
    assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)
    assert out[2].tolist() == starts.tolist()


@pytest.mark.parametrize("in_place", [False, True])
def test_tokens_without_an_entry_are_not_cached(gb, in_place):
    for tokens in (1, 6, 7, 99, 100, 101, 120, 150, 151, 209, 210):
        run_cut(gb, [10, 20, 30], [100, 50, 60], 16, 20, 40, tokens, in_place)
    # behind the last entry: a sequence that needs no page, one with no tokens
    run_cut(gb, [0, 1, 32, 15], [20, 3, 0, 1], 16, 4, 9, 20, in_place)
    rng = np.random.default_rng(4)
    for B, top in ((4096, 9), (513, 200), (3, 40000)):
        lens = [int(x) for x in rng.integers(0, 500, B)]
        new = [int(x) for x in rng.integers(0, top + 1, B)]
        for part in (0.1, 0.5, 0.99):
            run_cut(gb, lens, new, 16, -(-(500 + top) // 16) + 1, sum(new) // 16 + B + 5,
                    max(1, int(part * sum(new))), in_place, seed=B)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens", [3, 4, 12, 13, 15, 17, 18])
def test_rejected_sequences_keep_their_places_in_a_cut(gb, tokens, in_place):
    """A request whose row is full in the middle: the others' tokens stay where they were packed."""
    lens, new, page, width = [16, 160, 10], [4, 9, 5], 16, 10
    table, stack, pages, P = make([16, 0, 10], page, 9, width, 8)
    kept = entries(new, tokens)
    good = [0, 2]
    rt, rl, rs, _, _ = OT.extend(table[good], [16, 10], [kept[b] for b in good], stack, page)
    _, _, _, toks, _ = OT.extend(table[good], [16, 10], [4, 5], stack, page)
    gt, gl, gc = t(table), t(lens), t([len(stack)])
    kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
    out = gb.kv_paged_extend(gt, gl, t(new), t(pages), gc, page, P, max_tokens=tokens, **kw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    assert out[0].tolist() == [rl[0], 160, rl[1]] and out[1].item() == len(rs)
    got = gt.cpu().numpy()
    for row, b, n in zip(rt, good, held(rl, page)):
        assert np.array_equal(got[b, :n], row[:n])
    pos, slots, starts = OT.packed([toks[0], ([-1] * 9,) * 2, toks[1]], tokens)
    assert out[2].tolist() == starts.tolist()
    assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)


@pytest.mark.parametrize("in_place", [False, True])
def test_too_few_pages_and_entries(gb, in_place):
    """Behind a sequence that gets no pages, one that needs none, and the end of the entries."""
    lens, new, page, width = [16, 0, 30, 8], [20, 60, 2, 7], 16, 8
    table, stack, pages, P = make(lens, page, 20, width, 9, free=3)    # 2 pages taken, 4 not there
    rt, rl, rs, toks, refused = OT.extend(table, lens, new, stack, page)
    assert refused == [1] and len(rs) == 1
    for tokens in (83, 85, 89):
        gt, gl, gc = t(table), t(lens), t([len(stack)])
        kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
        out = gb.kv_paged_extend(gt, gl, t(new), t(pages), gc, page, P, max_tokens=tokens, **kw)
        assert gb.device_status() == gb.DEV_NO_PAGES | (gb.DEV_BAD_LENGTH if tokens < 89 else 0)
        kept = entries(new, tokens)
        assert out[0].tolist() == [36, 0, 30 + kept[2], 8 + kept[3]] and out[1].item() == len(rs)
        pos, slots, starts = OT.packed(toks, tokens)
        assert out[2].tolist() == starts.tolist() and np.array_equal(gt.cpu().numpy(), rt)
        assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)


@pytest.mark.parametrize("in_place", [False, True])
def test_the_rest_comes_with_the_next_call(gb, in_place):
    """What had no entry is brought again: every page is held once, and all of them come back."""
    lens, new, page, width = [10, 20, 30], [100, 50, 60], 16, 20
    table, stack, pages, P = make(lens, page, 40, width, 7)
    gt, gl, gp, gc = t(table), t(lens), t(pages), t([len(stack)])
    left = list(new)
    for tokens in (120, 45, 200):
        kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
        gl, gc, *_ = gb.kv_paged_extend(gt, gl, t(left), gp, gc, page, P, max_tokens=tokens, **kw)
        left = [m - k for m, k in zip(left, entries(left, tokens))]
        assert gb.device_status() == (gb.DEV_BAD_LENGTH if sum(left) else 0)
        assert gl.tolist() == [n + m - x for n, m, x in zip(lens, new, left)]
        got = gt.cpu().numpy()
        mine = [p for b, n in enumerate(held(gl.tolist(), page)) for p in got[b, :n].tolist()]
        assert sorted(mine + gp.tolist()[:gc.item()]) == list(range(P))
    assert left == [0, 0, 0]
    gc = gb.kv_paged_release(gt, gl, gp, gc, page, P)
    assert gb.device_status() == 0 and sorted(gp.tolist()[:gc.item()]) == list(range(P))
