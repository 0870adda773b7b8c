"""Pins for the oracle's FP16 page cache and differential attention (CPU only): brute force with
``math.exp`` over page walks, closed forms, and planted mistakes that a pin has to catch."""

import math

import numpy as np
import pytest

from attention_fp16_flashattention_gb300 import inputs
from oracle import attention as OA
from oracle import diff as OD
from oracle import paged as OP


def _brute_decode(q, kp, vp, table, lens, scale):
    """o and received weights by plain loops and math.exp without a max subtraction."""
    B, Hq, nq, D = q.shape
    ps, Hkv = kp.shape[1], kp.shape[2]
    o = np.zeros((B, Hq, nq, D))
    got = [np.zeros((Hkv, int(n))) for n in lens]
    for b in range(B):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            for i in range(nq):
                seen = [s for s in range(int(lens[b])) if s <= lens[b] - nq + i]
                e = {s: math.exp(scale * sum(float(x) * float(y) for x, y in zip(
                    q[b, h, i], kp[table[b, s // ps], s % ps, hk]))) for s in seen}
                total = sum(e.values())
                for s in seen:
                    got[b][hk, s] += e[s] / total
                    o[b, h, i] += e[s] / total * vp[table[b, s // ps], s % ps, hk].astype(float)
    return o, got


@pytest.mark.parametrize("Hq,Hkv,nq", [(4, 2, 1), (3, 1, 2), (2, 2, 3)])
def test_decode_brute_force(Hq, Hkv, nq):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(3, Hq, Hkv, nq, (37, 2, 0), 16, 1,
                                                        page_size=16, spare_pages=1, poison=True)
    ref = OP.decode(q, kp, vp, table, lens, 0.25)
    o, got = _brute_decode(q, kp, vp, table, lens, 0.25)
    assert np.allclose(ref["o"], o, atol=1e-12)
    for a, b in zip(ref["received"], got):
        assert np.allclose(a, b, atol=1e-12)
    rows = Hq // Hkv * nq
    assert np.isclose(ref["received"][0].sum(), rows * Hkv)      # every row hands out one in all
    assert np.all(np.isneginf(ref["lse"][2])) and np.all(ref["o"][2] == 0)


def test_decode_matches_causal_rows_of_the_dense_oracle():
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(1, 2, 1, 2, (50,), 32, 2, page_size=16)
    ref = OP.decode(q, kp, vp, table, lens, 0.2)
    k, v = (OP.slot_rows(x, table[0], 50)[:, 0].astype(np.float64) for x in (kp, vp))
    see = np.arange(50)[None, :] <= 48 + np.arange(2)[:, None]
    for h in range(2):
        o, lse = OA.attention_rows(q[0, h].astype(np.float64), k, v, 0.2, see)
        assert np.allclose(ref["o"][0, h], o) and np.allclose(ref["lse"][0, h], lse)


def test_append_then_read_back():
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 1, 2, 1, (40, 33), 8, 3, page_size=16)
    kn, vn = np.random.default_rng(1).standard_normal((2, 2, 2, 5, 8)).astype(np.float16)
    k2, v2, w2 = OP.append(kn, vn, kp, vp, table, lens, np.array([5, 2]), w)
    for b, c in ((0, 5), (1, 2)):
        n = lens[b]
        rows = OP.slot_rows(k2, table[b], n)
        assert np.array_equal(rows[n - c:], kn[b, :, :c].transpose(1, 0, 2))
        assert np.array_equal(rows[:n - c], OP.slot_rows(kp, table[b], n)[:n - c])
        assert np.array_equal(OP.slot_rows(v2, table[b], n)[n - c:], vn[b, :, :c].transpose(1, 0, 2))
    assert (w2 == 0).sum() == 2 * 7 and np.array_equal(w2[w2 != 0], w[w2 != 0])


def test_evict_kept_by_hand():
    w = np.array([9, 1, 5, 5, 7, 5, 2, 3], dtype=np.float32)
    assert OP.evict_kept(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert OP.evict_kept(w, 8, 4, 0, 0).tolist() == [0, 2, 3, 4]       # 9, 7, then two of three 5s
    assert OP.evict_kept(w, 8, 4, 2, 1).tolist() == [0, 1, 4, 7]
    assert OP.evict_kept(w, 8, 3, 0, 3).tolist() == [5, 6, 7]
    w[[4, 2]] = np.nan, -np.inf
    assert OP.evict_kept(w, 8, 6, 0, 0).tolist() == [0, 1, 3, 5, 6, 7]
    assert OP.evict_kept(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 5, 6, 7]
    assert OP.evict_kept(np.array([0.0, -0.0, 0.0]), 3, 2, 0, 0).tolist() == [0, 1]


def test_evict_rows_and_weights_travel_together():
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 1, 2, 1, (60, 20), 8, 4, page_size=16)
    k2, v2, w2, nl, kept = OP.evict(kp, vp, w, table, table, lens, 24, 2, 4)
    assert nl.tolist() == [24, 20]
    rows, old = OP.slot_rows(k2, table[0], 24), OP.slot_rows(kp, table[0], 60)
    for h in range(2):
        assert np.array_equal(rows[:, h], old[kept[0, h], h])
        assert kept[0, h, :2].tolist() == [0, 1] and kept[0, h, -4:].tolist() == [56, 57, 58, 59]
    assert np.array_equal(OP.slot_rows(k2, table[1], 20), OP.slot_rows(kp, table[1], 20))


def test_lambdas_closed_form():
    vecs = np.zeros((4, 3, 2))
    vecs[0, 1], vecs[1, 1] = [math.log(2), 0], [1, 5]
    assert np.allclose(OD.lambdas(vecs, 0.25, 3), [0.25, 1.25, 0.25])
    assert np.allclose(OD.lambdas(vecs[:, 1:2], 0.25, 3), 1.25)


def test_diff_brute_force_and_planted_mistakes():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((1, 2, 4, 8)), rng.standard_normal((1, 1, 6, 8)), \
        rng.standard_normal((1, 1, 6, 8))
    vecs = 0.3 * rng.standard_normal((4, 2, 4))
    g = 1 + 0.1 * rng.standard_normal(8)
    ref = OD.prefill(q, k, v, vecs, 0.4, 0.5, g, eps=1e-3)

    def brute(skip_norm=False, swap=False, shift=0):
        out = np.zeros((2, 4, 8))
        for h in range(2):
            lam = math.exp(sum(vecs[0, h] * vecs[1, h])) - math.exp(sum(vecs[2, h] * vecs[3, h])) + 0.4
            for i in range(4):
                seen = range(6 - 4 + i + 1 + shift)
                maps = []
                for part in (slice(0, 4), slice(4, 8)):
                    e = [math.exp(0.5 * float(q[0, h, i, part] @ k[0, 0, s, part])) for s in seen]
                    maps.append([x / sum(e) for x in e])
                if swap:
                    maps.reverse()
                o = sum((a - lam * c) * v[0, 0, s] for s, a, c in zip(seen, *maps))
                if not skip_norm:
                    o = o / math.sqrt(float(np.mean(o * o)) + 1e-3) * g * 0.6
                out[h, i] = o
        return out
    assert np.allclose(ref["o"][0], brute(), atol=1e-12)
    assert np.allclose(OD.prefill(q, k, v, vecs, 0.4, 0.5)["o"][0], brute(True), atol=1e-12)
    for wrong in (brute(True), brute(swap=True), brute(shift=-1)):
        assert not np.allclose(ref["o"][0], wrong, atol=1e-3)


def test_diff_lengths_and_decode_agree():
    rng = np.random.default_rng(6)
    q = rng.standard_normal((2, 2, 5, 8)).astype(np.float16)
    kp, vp = rng.standard_normal((2, 4, 16, 1, 8)).astype(np.float16)
    table, lens = np.array([[2, 0], [3, 1]]), np.array([20, 3])
    vecs = 0.1 * rng.standard_normal((4, 1, 4))
    dec = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.3, 0.5)
    k = np.stack([OP.slot_rows(kp, r, 32) for r in table]).transpose(0, 2, 1, 3)
    v = np.stack([OP.slot_rows(vp, r, 32) for r in table]).transpose(0, 2, 1, 3)
    pre = OD.prefill(q, k, v, vecs, 0.3, 0.5, q_lens=[5, 5], kv_lens=lens)
    assert np.allclose(dec["o"], pre["o"]) and np.array_equal(dec["lse"], pre["lse"])
    assert np.all(dec["o"][1, :, :2] == 0) and np.all(np.isneginf(dec["lse"][1, :, :, :2]))
    cut = OD.prefill(q, k, v, vecs, 0.3, 0.5, q_lens=[3, 0], kv_lens=lens)
    assert np.all(cut["o"][0, :, 3:] == 0) and np.all(cut["o"][1] == 0)
