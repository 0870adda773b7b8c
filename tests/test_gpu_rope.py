"""Per-head norms and rotary positions (qk_norm_rope_f16, kv_paged_rope_append) against float64.

Bounds.  A norm's factor: D squares summed in FP32 by eight and then in a tree (at most 13 roundings,
half of their relative error after the root), the mean and eps (2), rsqrtf (2 ulp, 2^-22), times the
weight and the element (2): below 2^-20.  An angle is known to 2^-32 of a turn and rounded to 24 bits of half
a turn, 2^-23 radians together, the sine and cosine to an ulp, 2^-23; two products and their sum round
three times.  So an output is off by less than 2^-19 of |a| + |b|, the two elements that it is made of,
before its last rounding: half a step of FP16 (2^-11 of itself, 2^-25 below its normal range) or of E4M3
(2^-4, 2^-10).
"""

import numpy as np
import pytest
import torch

from oracle import e4m3 as OE, rope as OR

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -19


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def close(got, ref, size, what, step=2.0 ** -11, least=2.0 ** -25):
    got = np.asarray(got, dtype=np.float64)
    excess = np.abs(got - ref) - (step * np.abs(ref) + least + E * size)
    assert np.all(excess <= 0), (f"{what}: {int((~(excess <= 0)).sum())} of {excess.size} outside, "
                                 f"worst {np.nanmax(excess):.3e}")


def inputs_of(B, Hq, Hk, S, D, rot, axes, norm, far, seed):
    rng = np.random.default_rng(seed)
    q, k, v = (rng.standard_normal((B, h, S, D)).astype(np.float16) * np.float16(1.5)
               for h in (Hq, Hk, Hk))
    pos = rng.integers(0, far + 1, (axes, B, S)).astype(np.int32)
    freqs = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    w = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    sections = None
    if axes > 1:
        cut = sorted(rng.integers(0, rot // 2 + 1, axes - 1).tolist())
        sections = np.diff([0] + cut + [rot // 2]).tolist()
    return q, k, v, pos, freqs, w, sections


CASES = [  # B, Hq, Hk, S, D, rot, axes, interleaved, norm, far
    (1, 1, 1, 1, 64, 64, 1, False, True, 10), (1, 1, 1, 1, 128, 128, 1, True, False, 10 ** 6),
    (2, 3, 1, 5, 64, 32, 1, True, True, 5000), (2, 3, 1, 5, 64, 8, 2, False, True, 2 ** 31 - 1),
    (3, 4, 2, 133, 128, 128, 1, False, True, 131071), (3, 4, 2, 133, 128, 64, 3, True, False, 70),
    (1, 6, 1, 77, 256, 256, 1, True, True, 2 ** 20), (1, 6, 1, 77, 256, 64, 1, False, False, 2 ** 20),
    (2, 5, 5, 40, 256, 40, 3, False, True, 300), (64, 32, 8, 1, 128, 128, 1, False, True, 8000),
    (1, 24, 24, 700, 128, 128, 3, False, True, 63), (1, 2, 2, 9000, 64, 56, 1, False, True, 9000),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_prompts(gb, case):
    B, Hq, Hk, S, D, rot, axes, inter, norm, far = case
    q, k, _, pos, freqs, w, sections = inputs_of(B, Hq, Hk, S, D, rot, axes, norm, far, S)
    go, gk = gb.qk_norm_rope_f16(t(q), t(k), t(pos if axes > 1 else pos[0]), t(freqs), q_weight=t(w[0]),
                                 k_weight=t(w[1]), eps=1e-5, interleaved=inter, sections=sections,
                                 rope_scale=1.25)
    assert gb.device_status() == 0
    for got, x, weight, what in ((go, q, w[0], "q"), (gk, k, w[1], "k")):
        ref, size = OR.rotate(x, pos, freqs, weight, 1e-5, inter, sections, 1.25)
        close(got.cpu().numpy(), ref, size, what)


def test_parts_left_out(gb):
    """One norm only, no rotation, no keys; what nothing is done to comes back bit for bit."""
    q, k, _, pos, freqs, w, _ = inputs_of(2, 3, 2, 9, 128, 64, 1, True, 100, 1)
    tq, tk, tw = t(q), t(k), t(w[0])
    go, gk = gb.qk_norm_rope_f16(tq, tk, None, None)
    assert torch.equal(go, tq) and torch.equal(gk, tk)
    go, gk = gb.qk_norm_rope_f16(tq, tk, t(pos[0]), None, q_weight=tw)
    close(go.cpu().numpy(), *OR.rotate(q, pos, None, w[0]), "norm")
    assert torch.equal(gk, tk)
    go, gk = gb.qk_norm_rope_f16(tq, None, t(pos[0]), t(freqs), k_weight=tw)
    assert gk is None
    close(go.cpu().numpy(), *OR.rotate(q, pos, freqs), "q alone")
    assert torch.equal(go[..., 64:], tq[..., 64:])
    zero = torch.zeros((2, 9), dtype=torch.int32, device=DEV)
    go, _ = gb.qk_norm_rope_f16(tq, tk, zero, t(freqs))
    assert torch.equal(go, tq)                         # position 0 turns nothing
    z = torch.zeros_like(tq)                           # a row of zeros has a norm all the same
    go, _ = gb.qk_norm_rope_f16(z, None, t(pos[0]), t(freqs), q_weight=tw)
    assert torch.equal(go, z) and gb.device_status() == 0


def test_infinite_and_nan_rows_stay_apart(gb):
    q, _, _, pos, freqs, w, _ = inputs_of(1, 2, 1, 6, 64, 64, 1, True, 9, 2)
    bad = q.copy()
    bad[0, 0, 1, 3], bad[0, 1, 4, 60] = np.inf, np.nan
    one, _ = gb.qk_norm_rope_f16(t(q), None, t(pos[0]), t(freqs), q_weight=t(w[0]))
    two, _ = gb.qk_norm_rope_f16(t(bad), None, t(pos[0]), t(freqs), q_weight=t(w[0]))
    one, two = one.cpu().numpy(), two.cpu().numpy()
    rows = np.ones((2, 6), dtype=bool)
    rows[0, 1] = rows[1, 4] = False
    assert np.array_equal(one[0][rows], two[0][rows])
    assert np.isnan(two[0, 0, 1, 3]) and np.isnan(two[0, 1, 4]).all()


def packed(q, k, v):
    """Views of one tensor [B][S][heads][D], as a model's projection leaves it."""
    heads = [x.shape[1] for x in (q, k, v)]
    whole = t(np.concatenate([q, k, v], 1).transpose(0, 2, 1, 3))
    return whole, [x.permute(0, 2, 1, 3) for x in whole.split(heads, 2)]


@pytest.mark.parametrize("B,S", [(1, 37), (3, 1), (2, 8), (1, 1)])
def test_in_place_in_a_packed_tensor(gb, B, S):
    """q and k of a packed projection are rotated where they lie; v between them stays."""
    q, k, v, pos, freqs, w, _ = inputs_of(B, 4, 2, S, 128, 128, 1, True, 500, 3)
    whole, (tq, tk, tv) = packed(q, k, v)
    wq, wk = t(w[0]), t(w[1])
    want = gb.qk_norm_rope_f16(tq, tk, t(pos[0]), t(freqs), q_weight=wq, k_weight=wk)
    out = gb.qk_norm_rope_f16(tq, tk, t(pos[0]), t(freqs), q_weight=wq, k_weight=wk, q_out=tq, k_out=tk)
    assert out[0] is tq and out[1] is tk
    assert torch.equal(tq, want[0]) and torch.equal(tk, want[1]) and torch.equal(tv, t(v))
    with pytest.raises(gb.GbattnError):                # k where q lies
        gb.qk_norm_rope_f16(tq, tk, t(pos[0]), t(freqs), k_out=tq[:, :2])
    with pytest.raises(gb.GbattnError):                # half a head further
        gb.qk_norm_rope_f16(tq[:, :3], None, t(pos[0]), t(freqs), q_out=tq[:, 1:4])


def test_padding_is_left_alone(gb):
    q, k, v, pos, freqs, w, _ = inputs_of(2, 3, 1, 21, 64, 64, 2, True, 50, 4)
    pos[0, 0, 5:9] = -1
    pos[1, 1, 20] = -2 ** 31
    skip = (pos < 0).any(0)
    outs = [torch.full(x.shape, 9.0, dtype=torch.float16, device=DEV) for x in (q, k)]
    gb.qk_norm_rope_f16(t(q), t(k), t(pos), t(freqs), q_weight=t(w[0]), sections=[16, 16], q_out=outs[0],
                        k_out=outs[1])
    for got, x, weight in ((outs[0], q, w[0]), (outs[1], k, None)):
        got = got.cpu().numpy().transpose(0, 2, 1, 3)
        ref, size = (y.transpose(0, 2, 1, 3) for y in OR.rotate(x, pos, freqs, weight, sections=[16, 16]))
        assert (got[skip] == 9).all()
        close(got[~skip], ref[~skip], size[~skip], "live rows")
    assert gb.device_status() == 0


# ---------------------------------------------------------------- into a cache

def run_append(gb, B, Hq, Hkv, S, D, rot, page, inter, norm, far, e4m3, seed, weights=True, pad=0.2,
               as_packed=True):
    q, k, v, pos, freqs, w, _ = inputs_of(B, Hq, Hkv, S, D, rot, 1, norm, far, seed)
    rng = np.random.default_rng(seed + 1)
    P = -(-B * S // page) + 2
    slots = rng.permutation(P * page)[:B * S].astype(np.int32).reshape(B, S)
    dead = rng.random((B, S)) < pad
    slots[dead] = rng.choice([-1, -5, -2 ** 31], int(dead.sum()))
    shape = (P, page, Hkv, D)
    kp, vp = (rng.integers(0, 127, shape).astype(np.uint8) if e4m3 else
              rng.standard_normal(shape).astype(np.float16) for _ in range(2))
    weight = rng.random((P, Hkv, page)).astype(np.float32)
    ks, vs = (0.11, 0.0625) if e4m3 else (3.0, 5.0)    # FP16 pages are not scaled
    tq, tk, tv = packed(q, k, v)[1] if as_packed else (t(q), t(k), t(v))
    gk, gv, gw = t(kp), t(vp), t(weight) if weights else None
    out = torch.full((B, Hq, S, D), 9.0, dtype=torch.float16, device=DEV)
    got = gb.kv_paged_rope_append(tq, tk, tv, t(slots), gk, gv, t(pos[0]), t(freqs), q_weight=t(w[0]),
                                  k_weight=t(w[1]), interleaved=inter, k_scale=ks, v_scale=vs,
                                  weights=gw, q_out=out)
    assert got is out and gb.device_status() == 0
    ref, size = OR.rotate(q, pos, freqs, w[0], interleaved=inter)
    alive = ~dead
    out = out.cpu().numpy().transpose(0, 2, 1, 3)
    assert (out[dead] == 9).all()
    close(out[alive], ref.transpose(0, 2, 1, 3)[alive], size.transpose(0, 2, 1, 3)[alive], "q")
    ref, size = (x.transpose(0, 2, 1, 3)[alive] for x in OR.rotate(k, pos, freqs, w[1], interleaved=inter))
    at = slots[alive]
    rk, rv = gk.cpu().numpy().reshape(-1, Hkv, D), gv.cpu().numpy().reshape(-1, Hkv, D)
    new_v = v.transpose(0, 2, 1, 3)[alive]
    if e4m3:
        close(OE.e4m3fn_decode(rk[at]), np.clip(ref / ks, -448, 448), size / ks, "k codes", 2.0 ** -4,
              2.0 ** -10)
        want = torch.from_numpy(new_v).float().div(vs).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert np.array_equal(rv[at], want.view(torch.uint8).numpy())
    else:
        close(rk[at], ref, size, "k pages")
        assert np.array_equal(rv[at].view(np.uint16), new_v.view(np.uint16))
    rest = np.ones(P * page, dtype=bool)
    rest[at] = False
    for got, before in ((rk, kp), (rv, vp)):
        assert np.array_equal(got[rest], before.reshape(-1, Hkv, D)[rest])
    if weights:
        weight[at // page, :, at % page] = 0
        assert np.array_equal(gw.cpu().numpy(), weight)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (64, 16, True), (128, 128, False),
                                         (128, 64, True), (256, 256, True), (256, 64, False)])
def test_append(gb, D, rot, inter, e4m3):
    run_append(gb, 2, 6, 2, 50, D, rot, 16, inter, True, 3000, e4m3, D + rot)
    run_append(gb, 1, 1, 1, 1, D, rot, 64, inter, False, 10, e4m3, D + rot, weights=False, pad=0)
    run_append(gb, 17, 8, 1, 1, D, rot, 256, inter, True, 90, e4m3, D + rot, as_packed=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_long_packed_prompts(gb, e4m3):
    run_append(gb, 1, 5, 3, 6001, 128, 128, 32, False, True, 200000, e4m3, 7, pad=0.01)


def test_append_bad_slots(gb):
    """A slot past the pool: that token's query is written, its key and value are not."""
    q, k, v, pos, freqs, _, _ = inputs_of(1, 2, 1, 4, 64, 64, 1, False, 50, 8)
    kp = torch.zeros((3, 16, 1, 64), dtype=torch.float16, device=DEV)
    vp = torch.zeros_like(kp)
    slots = t(np.array([[47, 48, 2 ** 31 - 1, 0]], dtype=np.int32))
    out = gb.kv_paged_rope_append(t(q), t(k), t(v), slots, kp, vp, t(pos[0]), t(freqs))
    assert gb.device_status() == gb.DEV_BAD_PAGE
    close(out.cpu().numpy(), *OR.rotate(q, pos, freqs), "q")
    rows = vp.reshape(48, 64).cpu().numpy()
    assert np.array_equal(rows[47], v[0, 0, 0]) and np.array_equal(rows[0], v[0, 0, 3])
    assert not rows[1:47].any() and not kp.reshape(48, 64)[1:47].any()


def test_e4m3_range_and_nan(gb):
    """Values beyond 448 scales become the largest code, NaN stays one."""
    v = np.zeros((1, 1, 1, 64), dtype=np.float16)
    v[..., :6] = [500, -65504, np.inf, -np.inf, np.nan, 1.0]
    kp = torch.zeros((1, 16, 1, 64), dtype=torch.uint8, device=DEV)
    vp = torch.zeros_like(kp)
    gb.kv_paged_rope_append(t(v), t(v), t(v), t(np.zeros((1, 1), dtype=np.int32)), kp, vp, None, None)
    for pages in (kp, vp):
        code = pages[0, 0, 0].cpu().numpy()
        assert code[:4].tolist() == [0x7E, 0xFE, 0x7E, 0xFE] and code[4] & 0x7F == 0x7F
        assert code[5] == 0x38 and not code[6:].any()


def test_graph_and_side_stream(gb):
    q, k, v, pos, freqs, w, _ = inputs_of(4, 8, 2, 3, 128, 128, 1, True, 700, 9)
    kp = torch.zeros((2, 16, 2, 128), dtype=torch.float16, device=DEV)
    vp = torch.zeros_like(kp)
    slots = t(np.arange(12, dtype=np.int32).reshape(4, 3))
    tq, tk, tv, tp, tf, tw = t(q), t(k), t(v), t(pos[0]), t(freqs), t(w[0])
    want = gb.kv_paged_rope_append(tq, tk, tv, slots, kp, vp, tp, tf, q_weight=tw)
    wk, wv = kp.clone(), vp.clone()
    kp.zero_(), vp.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = gb.kv_paged_rope_append(tq, tk, tv, slots, kp, vp, tp, tf, q_weight=tw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kp, wk) and torch.equal(vp, wv)
    out = gb.kv_paged_rope_append(tq, tk, tv, slots, kp, vp, tp, tf, q_weight=tw, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and gb.device_status() == 0


def test_pool_past_32_bit_offsets(gb):
    """Slots whose element offsets pass 2^32."""
    P, page, Hkv, D = 40000, 64, 8, 256
    kp = torch.empty((P, page, Hkv, D), dtype=torch.uint8, device=DEV)
    vp = torch.empty_like(kp)
    q, k, v, pos, freqs, _, _ = inputs_of(1, 1, Hkv, 2, D, 64, 1, False, 50, 10)
    slots = t(np.array([[P * page - 1, 2 ** 21 + 17]], dtype=np.int32))
    small = [torch.empty((1, 16, Hkv, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    gb.kv_paged_rope_append(t(q), t(k), t(v), slots, kp, vp, t(pos[0]), t(freqs))
    gb.kv_paged_rope_append(t(q), t(k), t(v), t(np.array([[0, 1]], dtype=np.int32)), *small, t(pos[0]),
                            t(freqs))
    for big, ref in ((kp, small[0]), (vp, small[1])):
        rows = big.view(P * page, Hkv, D)
        assert torch.equal(rows[P * page - 1], ref[0, 0]) and torch.equal(rows[2 ** 21 + 17], ref[0, 1])
    assert gb.device_status() == 0
