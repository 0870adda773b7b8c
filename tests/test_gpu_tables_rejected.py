"""Page tables where some of a batch's lengths are rejected (kv_paged_extend): the other requests' tokens
stay where the caller packed them."""

import numpy as np
import pytest
import torch

from oracle import rope as OR, tables as OT
from tests.test_gpu_rope import close
from tests.test_gpu_tables import make, t

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run_rejected(gb, lens, new, bad, page, width, spare, tokens, in_place, places=None, seed=1):
    """Sequences `bad` are rejected, the others served; places: tokens that each takes among the packed
    ones (None: its new ones)."""
    B = len(lens)
    places = list(new) if places is None else places
    clean = [0 if b in bad else lens[b] for b in range(B)]
    table, stack, pages, P = make(clean, page, spare, width, seed)
    good = [b for b in range(B) if b not in bad]
    rt, rl, rs, toks, refused = OT.extend(table[good], [lens[b] for b in good], [new[b] for b in good], stack, page)
    assert not refused
    want_table, want_lens = table.copy(), list(lens)
    want_table[good] = rt
    per = [([-1] * places[b],) * 2 for b in range(B)]
    for b, n, tok in zip(good, rl, toks):
        want_lens[b], per[b] = n, tok
    gt, gl, gc = t(table), t(lens), t([len(stack)])
    kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
    out = gb.kv_paged_extend(gt, gl, t(new), t(pages), gc, page, P, max_tokens=tokens, **kw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    assert out[0].tolist() == want_lens and out[1].item() == len(rs)
    assert np.array_equal(gt.cpu().numpy(), want_table)
    pos, slots, starts = OT.packed(per, tokens)
    assert out[2].tolist() == starts.tolist()
    assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)


@pytest.mark.parametrize("in_place", [False, True])
def test_rejected_sequences_keep_their_places(gb, in_place):
    # rows of 160 slots: at its end; one token past it; a prompt longer than the row
    run_rejected(gb, [16, 160, 30, 5], [3, 1, 4, 2], [1], 16, 10, 9, 12, in_place)
    run_rejected(gb, [16, 30, 100, 10], [1, 0, 61, 5], [2], 16, 10, 9, 67, in_place)
    run_rejected(gb, [0, 3, 0], [7, 200, 20], [1], 16, 10, 9, 250, in_place)
    # cached lengths out of range
    run_rejected(gb, [16, -1, 161, 2 ** 31 - 1, 9], [2, 3, 4, 5, 6], [1, 2, 3], 16, 10, 9, 20, in_place)
    # nothing can have been packed by a negative length, or by one that neither the entries nor a row could hold
    run_rejected(gb, [16, 30, 10, 7], [1, -3, 2 ** 31 - 1, 5], [1, 2], 16, 10, 9, 9, in_place,
                 places=[1, 0, 0, 5])
    # nor, beside such a one, by lengths whose sum is above them
    run_rejected(gb, [16, 160, 10, 30], [4, 9, 5, -1], [1, 3], 16, 10, 9, 17, in_place, places=[4, 0, 5, 0])
    run_rejected(gb, [16, 160, 10, 30], [4, 9, 5, 33], [1, 3], 16, 2, 9, 17, in_place, places=[4, 0, 5, 0])


@pytest.mark.parametrize("in_place", [False, True])
def test_rejected_among_many(gb, in_place):
    rng = np.random.default_rng(2)
    for B, top in ((4096, 5), (600, 300), (40, 2000)):
        width = 80
        lens = [int(x) for x in rng.integers(0, 700, B)]
        new = [int(x) for x in rng.integers(0, min(top, 500) + 1, B)]
        bad = sorted({0, B - 1, *rng.integers(0, B, B // 9).tolist()})
        for b in bad:
            if b % 2:
                lens[b] = -1 - b
            else:
                lens[b], new[b] = 16 * width, max(1, new[b])
        run_rejected(gb, lens, new, bad, 16, width, sum(new) // 16 + B + 5, sum(new) + 3, in_place, seed=B)


def test_a_request_at_its_end_beside_others_in_the_cache(gb):
    """Packed tokens through kv_paged_rope_append: the neighbours of a request whose row is full get their
    own keys and values, it gets none."""
    rng = np.random.default_rng(3)
    Hq, Hkv, D, ps, width, P = 4, 2, 64, 16, 4, 24
    lens, new = [20, 64, 0, 47], [5, 1, 18, 1]
    table = np.full((4, width), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // ps)] = 4 * b + np.arange(-(-n // ps))
    stack = list(range(16, P))
    gt, T = t(table), sum(new)
    out, count, starts, pos, slots = gb.kv_paged_extend(gt, t(lens), t(new), t(stack), t([len(stack)]), ps, P,
                                                        max_tokens=T)
    assert gb.device_status() == gb.DEV_BAD_LENGTH and out.tolist() == [25, 64, 18, 48]
    q, k, v = (rng.standard_normal((1, h, T, D)).astype(np.float16) for h in (Hq, Hkv, Hkv))
    kp, vp = (torch.full((P, ps, Hkv, D), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
    freqs = gb.rope_frequencies(D)
    gb.kv_paged_rope_append(*(torch.from_numpy(x).to(DEV) for x in (q, k, v)), slots[None], kp, vp, pos[None], freqs)
    assert gb.device_status() == 0
    where = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)])
    turned, size = OR.rotate(k, where[None, None], freqs.cpu().numpy())
    table, kp, vp = gt.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy()
    written = np.zeros((P, ps), dtype=bool)
    for b, at in zip(range(4), np.cumsum([0] + new)):
        if b == 1:
            continue
        s = np.arange(lens[b], lens[b] + new[b])
        pages, off = table[b, s // ps], s % ps
        written[pages, off] = True
        rows = slice(at, at + new[b])
        assert np.array_equal(vp[pages, off], v[0, :, rows].transpose(1, 0, 2)), b
        close(kp[pages, off], turned[0, :, rows].transpose(1, 0, 2), size[0, :, rows].transpose(1, 0, 2), f"keys {b}")
    assert (kp[~written] == 7).all() and (vp[~written] == 7).all()
