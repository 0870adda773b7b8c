"""The FP16 page cache on the GPU: append, decode with accumulated weights, eviction, and a run
of the three as a serving loop uses them, against the float64 oracle.

Bounds.  With X the largest scale * sum_i |q_i k_i| of a row, an FP32 score is off by at most
D 2^-23 X (one truncating addition per product) plus its scaling's rounding, so a probability is
off by a relative e = 2 (D 2^-23 X + 2^-21) + 2^-20 (numerator, denominator, two exponentials of
two ulp each).  The hi + lo halves of P carry 2^-22 more, so
|o - ref| <= 2^-11 |ref| + 2^-25 + 2 e sum p|v| (half a step of FP16, its subnormals' half step,
P and the sums), |lse - ref| <= e + 2^-23 |ref|, and a received weight is off by e of itself,
plus half a step of the FP32 sum.
"""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def row_error(size, D):
    return 2 * (D * 2.0 ** -23 * size + 2.0 ** -21) + 2.0 ** -20


def assert_within(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    same_inf = np.isneginf(got) & np.isneginf(ref)
    with np.errstate(invalid="ignore"):
        excess = np.where(same_inf, -1.0, np.abs(got - ref) - tol)
    assert np.all(excess <= 0), (f"{what}: {int((~(excess <= 0)).sum())} of {excess.size} outside, "
                                 f"worst {np.nanmax(excess):.3e}")


def check_decode(gb, q, kp, vp, table, lens, w=None, scale=None, max_kv=None, workspace=None):
    """One decode call against the oracle; returns (o, weights) as numpy."""
    B, Hq, nq, D = q.shape
    scale = inputs.softmax_scale(D) if scale is None else scale
    lse = torch.full((B, Hq, nq), 7.0, device=DEV)
    tw = t(w)
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), max_kv_len=max_kv,
                                     lse=lse, weights=tw, scale=scale, workspace=workspace)
    assert gb.device_status() == 0
    ref = OP.decode(q, kp, vp, table, lens, scale)
    e = row_error(ref["size"], D)
    assert_within(o.float().cpu().numpy(), ref["o"],
                  2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], "o")
    with np.errstate(invalid="ignore"):
        assert_within(lse.cpu().numpy(), ref["lse"], e + 2.0 ** -23 * np.abs(ref["lse"]), "lse")
    if w is not None:
        ps = kp.shape[1]
        want, tol = w.astype(np.float64), np.zeros(w.shape)
        for b, n in enumerate(lens):
            s = np.arange(n)
            page = table[b, s // ps]
            for h in range(kp.shape[2]):
                want[page, h, s % ps] += ref["received"][b][h]
                tol[page, h, s % ps] += 2 * float(e.max()) * ref["received"][b][h] + 2.0 ** -100
        tol = np.where(tol > 0, tol + 2.0 ** -23 * np.abs(want), 0.0)   # untouched entries: exact
        assert_within(tw.cpu().numpy(), want, tol, "weights")
        return o, tw.cpu().numpy()
    return o, None


# ---------------------------------------------------------------- append

def run_append(gb, B, Hkv, n, D, ps, lens, new_lens=None, weights=True, token_major=False, seed=1):
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(B, Hkv, Hkv, 1, lens, D, seed,
                                                        page_size=ps, spare_pages=2)
    rng = np.random.default_rng(seed)
    kn, vn = rng.standard_normal((2, B, Hkv, n, D)).astype(np.float16)
    new = None if new_lens is None else np.asarray(new_lens, dtype=np.int32)
    tk, tv = t(kn), t(vn)
    if token_major:
        tk, tv = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (tk, tv))
    gk, gv, gw = t(kp), t(vp), t(w) if weights else None
    gb.kv_paged_append_f16(tk, tv, gk, gv, t(table), t(lens), new_lens=t(new), weights=gw)
    rk, rv, rw = OP.append(kn, vn, kp, vp, table, lens, new, w)
    assert gb.device_status() == 0
    assert np.array_equal(gk.cpu().numpy(), rk) and np.array_equal(gv.cpu().numpy(), rv)
    if weights:
        assert np.array_equal(gw.cpu().numpy(), rw)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_append_one_token(gb, D, ps, Hkv):
    run_append(gb, 4, Hkv, 1, D, ps, (1, 16, 17, 200), token_major=Hkv == 8)


@pytest.mark.parametrize("token_major", [False, True])
def test_append_ragged_prompts(gb, token_major):
    """Several tokens, some rows not appended, one sequence none at all."""
    run_append(gb, 4, 2, 133, 128, 32, (133, 300, 64, 150), new_lens=(133, 7, 0, 1),
               token_major=token_major)
    run_append(gb, 2, 5, 70, 64, 16, (70, 71), weights=False, token_major=token_major)


def test_append_bad_lengths_and_pages_are_skipped(gb):
    _, kp, vp, table, _, w = inputs.paged_f16_inputs(4, 1, 1, 1, (40, 40, 40, 40), 64, 3,
                                                     page_size=16)
    kn, vn = np.random.default_rng(4).standard_normal((2, 4, 1, 3, 64)).astype(np.float16)
    lens = np.array([2, 40, 49, 40], dtype=np.int32)     # fewer than the new ones; past the table
    bad = table.copy()
    bad[3, 2] = kp.shape[0]
    gk, gv, gw = t(kp), t(vp), t(w)
    gb.kv_paged_append_f16(t(kn), t(vn), gk, gv, t(bad), t(lens), weights=gw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH | gb.DEV_BAD_PAGE
    rk, rv, rw = OP.append(kn[1:2], vn[1:2], kp, vp, table[1:2], lens[1:2], None, w)
    assert np.array_equal(gk.cpu().numpy(), rk) and np.array_equal(gv.cpu().numpy(), rv)
    assert np.array_equal(gw.cpu().numpy(), rw)


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ps", [16, 64, 256])
def test_decode_widths_and_pages(gb, D, ps):
    """Ragged lengths down to one and none; NaN wherever no sequence holds a row."""
    case = inputs.paged_f16_inputs(5, 8, 2, 1, (1000, 1, 0, 333, 16), D, 11, page_size=ps,
                                   spare_pages=2, poison=True)
    check_decode(gb, *case)


@pytest.mark.parametrize("Hq,Hkv,nq", [(1, 1, 1), (6, 1, 1), (8, 1, 1), (9, 1, 1), (16, 2, 1),
                                       (12, 4, 5), (5, 5, 3), (16, 1, 2), (20, 1, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_head_layouts(gb, Hq, Hkv, nq, D):
    """Query rows below, at and above one MMA block and one row group; the causal tail of several
    new tokens; a sequence shorter than its new tokens (rows that see nothing)."""
    case = inputs.paged_f16_inputs(3, Hq, Hkv, nq, (517, max(nq - 2, 0), 90), D, 12, page_size=32,
                                   poison=True)
    check_decode(gb, *case)


@pytest.mark.parametrize("std", [0.05, 4.0])
def test_decode_flat_and_peaked_scores(gb, std):
    case = inputs.paged_f16_inputs(2, 8, 2, 1, (3000, 700), 128, 13, q_std=std)
    check_decode(gb, *case)


def test_decode_many_and_long_sequences(gb):
    """More sequences than threads, then one long sequence next to short ones."""
    lens = tuple(int(x) for x in np.random.default_rng(14).integers(0, 40, 700))
    check_decode(gb, *inputs.paged_f16_inputs(700, 2, 1, 1, lens, 64, 14, page_size=16))
    check_decode(gb, *inputs.paged_f16_inputs(3, 4, 1, 1, (70001, 3, 50), 128, 15, page_size=128))


@pytest.mark.parametrize("Hq,Hkv,nq", [(3, 3, 1), (9, 1, 1), (16, 2, 2), (20, 1, 2), (6, 2, 4)])
@pytest.mark.parametrize("D", [64, 256])
def test_decode_weights_over_row_groups(gb, Hq, Hkv, nq, D):
    """Weights summed over one row, one and several row groups; rows that see nothing add none."""
    case = inputs.paged_f16_inputs(4, Hq, Hkv, nq, (530, nq - 1, 33, 0), D, 22, page_size=16,
                                   spare_pages=1, poison=True)
    check_decode(gb, *case)


@pytest.mark.parametrize("Hq,D", [(32, 128), (20, 64), (64, 256), (100, 64)])
def test_decode_row_groups_side_by_side(gb, Hq, D):
    """A length bound above 256 MB of cache, where 2, 4 or 8 row groups share a CTA's tiles."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, Hq, 1, 1, (2100, 40, 700), D, 24,
                                                        page_size=64, poison=True)
    wide = np.zeros((3, 1 << 16), dtype=np.int32)       # 4M tokens of bound, the rest not in use
    wide[:, :table.shape[1]] = table
    case = (q, kp, vp, wide, lens)
    check_decode(gb, *case)
    lse = torch.empty((3, Hq, 1), device=DEV)
    n = gb.attn_paged_decode_f16_workspace_size(3, Hq, 1, 1, 400000, D, True)
    tw = t(w)
    o = gb.attn_paged_decode_f16_fwd(*(t(x) for x in case), max_kv_len=400000, lse=lse, weights=tw,
                                     workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    narrow = t(w)
    want = gb.attn_paged_decode_f16_fwd(*(t(x) for x in (q, kp, vp, table, lens)), weights=narrow)
    assert gb.device_status() == 0
    assert (o.float() - want.float()).abs().max().item() <= 2.0 ** -10    # other joins, same bounds
    assert torch.allclose(tw, narrow, rtol=1e-5, atol=1e-6)
    check_decode(gb, *case, w=w, max_kv=400000)


def test_decode_most_sequences(gb):
    """4096 sequences, the most a call takes, some of them empty, with the narrow and the wide CTA."""
    lens = tuple(int(x) for x in np.random.default_rng(23).integers(0, 5, 4096))
    for D in (64, 256):
        check_decode(gb, *inputs.paged_f16_inputs(4096, 1, 1, 1, lens, D, 23, page_size=16))


@pytest.mark.parametrize("Hq,Hkv,nq", [(1, 1, 1), (6, 1, 2), (16, 2, 2), (20, 1, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_kv", [None, 300000])
def test_decode_short_caches_both_ways(gb, Hq, Hkv, nq, D, max_kv):
    """Lengths from none to 700, in clusters of eight CTAs a stream down to one, and under a bound so
    far above them that the streams' tiles are laid end to end."""
    for lens in ((700,), (1, 0, 17, 300), tuple(range(40)), tuple(range(5, 300, 4))):
        q, kp, vp, table, lens, w = inputs.paged_f16_inputs(len(lens), Hq, Hkv, nq, lens, D, 50,
                                                            page_size=16, poison=True)
        if max_kv is not None:
            wide = np.full((len(lens), max_kv // 16), -1, dtype=np.int32)
            wide[:, :table.shape[1]] = table
            table = wide
        check_decode(gb, q, kp, vp, table, lens, max_kv=max_kv)
        check_decode(gb, q, kp, vp, table, lens, w, max_kv=max_kv)


def test_decode_bad_length_in_clusters(gb):
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, 4, 2, 1, (90, 100, 50), 64, 51, page_size=16)
    bad, bad_lens = table.copy(), lens.copy()
    bad[0, 2] = -7
    bad_lens[2] = 5000
    tw, lse = t(w), torch.zeros((3, 4, 1), device=DEV)
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(bad), t(bad_lens), lse=lse, weights=tw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH | gb.DEV_BAD_PAGE
    assert torch.all(o[2] == 0) and torch.all(torch.isneginf(lse[2]))
    ref = OP.decode(q[1:2], kp, vp, table[1:2], lens[1:2], inputs.softmax_scale(64))
    assert np.abs(o[1].float().cpu().numpy() - ref["o"][0]).max() < 2e-3
    gone = np.concatenate([table[0, 2:3], table[2, :4]])   # the bad page's tokens, the bad length's
    assert np.array_equal(tw.cpu().numpy()[gone], w[gone])


def test_decode_smaller_workspace_and_refusals(gb):
    case = inputs.paged_f16_inputs(2, 8, 2, 1, (3000, 700), 128, 16)
    full = gb.attn_paged_decode_f16_workspace_size(2, 8, 2, 1, 3008, 128, True)
    scores = full - gb.attn_paged_decode_f16_workspace_size(2, 8, 2, 1, 3008, 128, False)
    a, _ = check_decode(gb, *case)
    for part in (3, 15):   # 160 records in all; one CTA and four streams need 9
        ws = torch.empty(scores + (full - scores) // part, dtype=torch.uint8, device=DEV)
        check_decode(gb, *case, workspace=ws)
    with pytest.raises(gb.GbattnError):
        check_decode(gb, *case, workspace=torch.empty(scores, dtype=torch.uint8, device=DEV))


def test_decode_garbage_workspace_and_repeats(gb):
    """The workspace's contents do not matter, and two calls give the same bits."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, 8, 2, 2, (3000, 700, 40), 128, 17)
    n = gb.attn_paged_decode_f16_workspace_size(3, 8, 2, 2, table.shape[1] * 32, 128, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    a, wa = check_decode(gb, q, kp, vp, table, lens, w, workspace=ws)
    b, wb = check_decode(gb, q, kp, vp, table, lens, w, workspace=ws)
    assert torch.equal(a, b) and np.array_equal(wa, wb)


def test_decode_bad_length_and_page(gb):
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, 4, 2, 1, (200, 100, 50), 64, 18,
                                                        page_size=16)
    bad, bad_lens = table.copy(), lens.copy()
    bad[0, 2] = kp.shape[0] + 9
    bad_lens[2] = -1
    tw, lse = t(w), torch.zeros((3, 4, 1), device=DEV)
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(bad), t(bad_lens), lse=lse, weights=tw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH | gb.DEV_BAD_PAGE
    assert torch.all(o[2] == 0) and torch.all(torch.isneginf(lse[2]))
    ref = OP.decode(q[1:2], kp, vp, table[1:2], lens[1:2], inputs.softmax_scale(64))
    assert np.abs(o[1].float().cpu().numpy() - ref["o"][0]).max() < 2e-3
    untouched = table[2, :4]
    assert np.array_equal(tw.cpu().numpy()[untouched], w[untouched])


def test_decode_shared_prefix_pages_add_up(gb):
    """Two sequences over the same first pages: both add to the shared weights."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 4, 1, 1, (64, 64), 64, 19, page_size=16)
    table[1, :2] = table[0, :2]
    check_decode(gb, q, kp, vp, table, lens, w)


def test_decode_on_another_stream_and_in_a_graph(gb):
    """A side stream without a workspace of its own, then a captured call replayed with new data
    in the same buffers."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 8, 2, 1, (900, 450), 128, 20)
    tq, tk, tv, tt, tl = t(q), t(kp), t(vp), t(table), t(lens)
    want = gb.attn_paged_decode_f16_fwd(tq, tk, tv, tt, tl)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = gb.attn_paged_decode_f16_fwd(tq, tk, tv, tt, tl, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    n = gb.attn_paged_decode_f16_workspace_size(2, 8, 2, 1, table.shape[1] * 32, 128, True)
    ws, o, tw = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty_like(tq), t(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.attn_paged_decode_f16_fwd(tq, tk, tv, tt, tl, o=o, weights=tw, workspace=ws)
    tl.copy_(t(np.array([77, 449], dtype=np.int32)))
    tq.mul_(0.5)
    tw.copy_(t(w))
    eager_w = t(w)
    want = gb.attn_paged_decode_f16_fwd(tq, tk, tv, tt, tl, weights=eager_w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(tw, eager_w)


def test_decode_abandoned_load_is_reported(gb):
    """A load that never arrives ends in the wait limit and the status word, and the next call is
    right again."""
    case = inputs.paged_f16_inputs(2, 8, 2, 1, (900, 450), 128, 21)
    q, kp, vp, table, lens, _ = case
    gb.set_wait_limit_ns(20_000_000)
    try:
        for mode in (1, 2):
            gb.test_inject_fault(mode)
            gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens))
            assert mode == 2 or gb.device_status() & gb.DEV_WAIT_TIMEOUT
            gb.device_status()
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    check_decode(gb, *case)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_decode_rows_that_see_nothing_beside_an_infinite_value(gb, D):
    """A query before the cache's first token gives O = 0 although a later query's value is inf."""
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(2, 4, 1, 5, (2, 700), D, 27)
    vp[table[0, 0], 0] = np.inf
    lse = torch.zeros((2, 4, 5), device=DEV)
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), lse=lse)
    assert gb.device_status() == 0
    assert torch.all(o[0, :, :3] == 0) and torch.all(torch.isneginf(lse[0, :, :3]))
    # a row that sees the inf is not finite; inf or NaN, since P = hi + lo with lo zero or negative
    # and 0 inf = NaN, inf - inf = NaN
    assert not torch.isfinite(o[0, :, 3:]).any() and torch.isfinite(o[1]).all()


def test_abandoned_loads_with_weights_touch_no_other_weight(gb):
    """A decode that gives up describes none of its tiles as live, whatever its workspace held: no
    weight outside the sequences' slots moves, and the next call is right again."""
    lens = (40000, 17)   # far more tiles than a warp fetches pages for in advance
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 4, 1, 1, lens, 64, 26, spare_pages=40)
    held = np.zeros(w.shape, dtype=bool)
    for b, n in enumerate(lens):
        at = np.arange(n)
        held[table[b, at // 32], :, at % 32] = True
    # one CTA's worth of workspace (a record: 8 rows of 64 values, a max and a sum), so that every
    # warp's range is long
    full = gb.attn_paged_decode_f16_workspace_size(2, 4, 1, 1, table.shape[1] * 32, 64, True)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ws = torch.empty(full - (sms - 1) * 8 * (64 * 4 + 8), dtype=torch.uint8, device=DEV)
    gb.set_wait_limit_ns(20_000_000)
    try:
        for mode in (1, 2):
            gb.test_inject_fault(mode)
            gw = t(w)
            ws.fill_(255)
            gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), weights=gw,
                                         workspace=ws)
            assert gb.device_status() & gb.DEV_WAIT_TIMEOUT
            assert np.array_equal(gw.cpu().numpy()[~held], w[~held])
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    check_decode(gb, q, kp, vp, table, lens, w, workspace=ws)


# ---------------------------------------------------------------- eviction

def run_evict(gb, lens, budget, sink=0, recent=0, Hkv=2, D=64, ps=16, in_place=True, seed=31,
              ties=False, bytes_=False, max_kv=None):
    B = len(lens)
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(B, Hkv, Hkv, 1, lens, D, seed, page_size=ps,
                                                        spare_pages=B * -(-budget // ps) + 1)
    if bytes_:
        kp, vp = (x.view(np.uint8)[..., ::2].copy() for x in (kp, vp))
    if ties:   # few distinct weights, zeros of both signs, NaN and infinities among them
        pick = np.random.default_rng(seed).integers(0, 7, w.shape)
        w = np.array([0.0, -0.0, 1.0, 2.0, np.nan, np.inf, -np.inf], dtype=np.float32)[pick]
    dst = table
    if not in_place:
        free = np.setdiff1d(np.arange(kp.shape[0]), table[table >= 0]).astype(np.int32)
        need = -(-budget // ps)
        dst = free[:B * need].reshape(B, need)
    gk, gv, gw = t(kp), t(vp), t(w)
    tt = t(table)
    new_lens, kept = gb.kv_paged_evict(gk, gv, gw, tt, t(lens), budget, sink=sink, recent=recent,
                                       dst_table=None if in_place else t(dst), max_kv_len=max_kv)
    assert gb.device_status() == 0
    rk, rv, rw, rl, rkept = OP.evict(kp, vp, w, table, dst, lens, budget, sink, recent)
    assert np.array_equal(new_lens.cpu().numpy(), rl)
    assert np.array_equal(kept.cpu().numpy(), rkept)
    view = np.uint16 if not bytes_ else np.uint8
    assert np.array_equal(gk.cpu().numpy().view(view), rk.view(view))
    assert np.array_equal(gv.cpu().numpy().view(view), rv.view(view))
    assert np.array_equal(gw.cpu().numpy().view(np.uint32), rw.view(np.uint32))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("budget,sink,recent", [(64, 4, 16), (64, 0, 0), (64, 0, 64), (64, 64, 0),
                                                (64, 20, 44), (1, 0, 0), (100, 3, 1)])
def test_evict_policies(gb, budget, sink, recent, in_place):
    """Lengths below, at and above the budget, one and none."""
    run_evict(gb, (500, 64, 65, 1, 0, 63, 130), budget, sink, recent, in_place=in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("D,ps,bytes_", [(64, 16, False), (128, 64, False), (256, 32, False),
                                         (256, 128, True), (64, 16, True)])
def test_evict_widths_and_ties(gb, D, ps, bytes_, ties, in_place):
    run_evict(gb, (700, 1300), 333, 5, 40, Hkv=3, D=D, ps=ps, bytes_=bytes_, ties=ties,
              in_place=in_place)


@pytest.mark.parametrize("lens,Hkv,budget", [((70000,), 1, 5000), ((30000, 1000), 2, 29000),
                                             (tuple([300] * 90), 2, 250),
                                             (tuple([120] * 200), 2, 100)])
def test_evict_cluster_sizes(gb, lens, Hkv, budget):
    """Grids that give a head eight CTAs, and down to one."""
    run_evict(gb, lens, budget, 4, 50, Hkv=Hkv, D=64, ps=64)


def test_evict_more_slots_than_the_key_array(gb):
    """One head of 215,000 slots: a CTA's share passes the keys it holds."""
    run_evict(gb, (215000,), 3000, 4, 1000, Hkv=1, D=64, ps=256, in_place=False)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("weights", ["equal", "one digit", "two digits", "ties"])
def test_evict_in_clusters_with_alike_weights(gb, weights, in_place):
    """The keys of the chosen first digit fill the lists of a cluster's CTAs, or pass them (from about
    13,000 on at these lengths)."""
    lens = (30000, 12000)
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 1, 1, 1, lens, 64, 47, page_size=64,
                                                        spare_pages=128)
    rng = np.random.default_rng(48)
    w = {"equal": np.full(w.shape, 0.25), "one digit": 1.0 + 0.2 * rng.random(w.shape),
         "two digits": np.where(rng.random(w.shape) < 0.5, 1.0 + 0.2 * rng.random(w.shape),
                                2.0 + 0.4 * rng.random(w.shape)),
         "ties": rng.integers(0, 4, w.shape)}[weights].astype(np.float32)
    spare = np.setdiff1d(np.arange(kp.shape[0]), table)[:128].reshape(2, 64).astype(np.int32)
    gk, gv, gw, tt = t(kp), t(vp), t(w), t(table)
    for budget in (4000, 3999):
        dst = table if in_place else spare
        new_lens, kept = gb.kv_paged_evict(gk, gv, gw, tt, t(lens), budget, sink=7, recent=100,
                                           dst_table=None if in_place else t(dst))
        assert gb.device_status() == 0
        kp, vp, w, rlens, rkept = OP.evict(kp, vp, w, table, dst, lens, budget, 7, 100)
        assert np.array_equal(kept.cpu().numpy(), rkept)
        assert np.array_equal(new_lens.cpu().numpy(), rlens)
        assert np.array_equal(gk.cpu().numpy(), kp) and np.array_equal(gv.cpu().numpy(), vp)
        assert np.array_equal(gw.cpu().numpy(), w)
        lens = rlens if in_place else lens


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("at", [0, 100, 150, 700, 839])   # sinks, held keys, beyond them, recent
def test_evict_bad_page_of_a_long_sequence(gb, at, in_place):
    """A page out of range anywhere in a sequence that eight CTAs share leaves it as it is."""
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 1, 1, 1, (215000, 500), 64, 49, page_size=256,
                                                        spare_pages=8)
    spare = np.setdiff1d(np.arange(kp.shape[0]), table)[:8].reshape(2, 4).astype(np.int32)
    bad = table.copy()
    bad[0, at] = kp.shape[0]
    dst = bad if in_place else spare
    gk, gv, gw, tt = t(kp), t(vp), t(w), t(bad)
    new_lens, kept = gb.kv_paged_evict(gk, gv, gw, tt, t(lens), 400, sink=30, recent=200,
                                       dst_table=None if in_place else t(dst))
    assert gb.device_status() == gb.DEV_BAD_PAGE
    rk, rv, rw, _, rkept = OP.evict(kp, vp, w, table[1:], dst[1:], lens[1:], 400, 30, 200)
    assert new_lens.cpu().tolist() == [215000, 400]
    assert torch.all(kept[0] == -1) and np.array_equal(kept[1:].cpu().numpy(), rkept)
    assert np.array_equal(gk.cpu().numpy(), rk) and np.array_equal(gv.cpu().numpy(), rv)
    assert np.array_equal(gw.cpu().numpy(), rw)


def test_evict_one_at_a_time(gb):
    """A step of a loop that evicts as soon as the budget is passed: most rows do not move."""
    run_evict(gb, (1025, 1024, 1026), 1024, 4, 64, Hkv=2, D=128, ps=16)


def test_evict_bad_sequences_stay(gb):
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(4, 1, 1, 1, (200, 200, 200, 200), 64, 33,
                                                        page_size=16)
    bad, bad_lens = table.copy(), lens.copy()
    bad[0, 12] = -1
    bad_lens[1], bad_lens[2] = -5, 209
    gk, gv, gw = t(kp), t(vp), t(w)
    new_lens, kept = gb.kv_paged_evict(gk, gv, gw, t(bad), t(bad_lens), 100, recent=10)
    assert gb.device_status() == gb.DEV_BAD_LENGTH | gb.DEV_BAD_PAGE
    rk, rv, rw, _, rkept = OP.evict(kp, vp, w, table[3:], table[3:], lens[3:], 100, 0, 10)
    assert new_lens.cpu().tolist() == [200, -5, 209, 100]
    assert torch.all(kept[:3] == -1) and np.array_equal(kept[3:].cpu().numpy(), rkept)
    assert np.array_equal(gk.cpu().numpy(), rk) and np.array_equal(gv.cpu().numpy(), rv)
    assert np.array_equal(gw.cpu().numpy(), rw)


def captured(call):
    """`call` captured into a graph and replayed once."""
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("in_place", [True, False])
def test_append_and_evict_in_graphs_and_on_a_side_stream(gb, in_place):
    """The same bits captured and replayed, and on a stream of its own, as called directly."""
    B, Hkv, D, ps, budget = 3, 2, 128, 16, 100
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(B, Hkv, Hkv, 1, (300, 90, 150), D, 34,
                                                        page_size=ps, spare_pages=B * 7)
    free = np.setdiff1d(np.arange(kp.shape[0]), table[table >= 0]).astype(np.int32)
    dst = None if in_place else t(free.reshape(B, 7))
    kn = np.random.default_rng(34).standard_normal((B, Hkv, 5, D)).astype(np.float16)
    tk, tt, tl = t(kn), t(table), t(lens)
    side, results = torch.cuda.Stream(), []
    for how in ("direct", "graph", "side"):
        gk, gv, gw = t(kp), t(vp), t(w)

        def step(stream=None):
            gb.kv_paged_append_f16(tk, tk, gk, gv, tt, tl, weights=gw, stream=stream)
            return gb.kv_paged_evict(gk, gv, gw, tt, tl, budget, sink=3, recent=20, dst_table=dst,
                                     stream=stream)
        torch.cuda.synchronize()
        out = captured(step) if how == "graph" else step(side if how == "side" else None)
        torch.cuda.synchronize()
        results.append([x.clone() for x in (gk, gv, gw) + tuple(out)])
    assert gb.device_status() == 0
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_evict_the_same_cache_twice(gb):
    """A second eviction right behind the first on the stream, on the lengths that the first wrote."""
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 2, 2, 1, (400, 310), 64, 35, page_size=16)
    gk, gv, gw, tt = t(kp), t(vp), t(w), t(table)
    l1, _ = gb.kv_paged_evict(gk, gv, gw, tt, t(lens), 200, sink=2, recent=30)
    l2, kept = gb.kv_paged_evict(gk, gv, gw, tt, l1, 77, sink=2, recent=30)
    k1, v1, w1, n1, _ = OP.evict(kp, vp, w, table, table, lens, 200, 2, 30)
    k2, v2, w2, n2, rkept = OP.evict(k1, v1, w1, table, table, n1, 77, 2, 30)
    assert np.array_equal(l2.cpu().numpy(), n2) and np.array_equal(kept.cpu().numpy(), rkept)
    assert np.array_equal(gk.cpu().numpy(), k2) and np.array_equal(gv.cpu().numpy(), v2)
    assert np.array_equal(gw.cpu().numpy(), w2) and gb.device_status() == 0


# ---------------------------------------------------------------- together

def test_serving_loop_with_a_budget(gb):
    """Prompt in, then steps of append + decode with weights, evicting whenever a cache passes its
    budget by a page: every step's output against the oracle on the oracle's own cache."""
    B, Hq, Hkv, D, ps, budget = 3, 8, 2, 64, 16, 48
    rng = np.random.default_rng(40)
    P = B * 6
    perm = rng.permutation(P).astype(np.int32).reshape(B, 6)
    kp = np.full((P, ps, Hkv, D), np.nan, dtype=np.float16)
    vp = kp.copy()
    w = np.full((P, Hkv, ps), 3.0, dtype=np.float32)
    gk, gv, gw, tt = t(kp), t(vp), t(w), t(perm)
    lens = np.zeros(B, dtype=np.int32)
    scale = inputs.softmax_scale(D)

    def feed(n, new_lens):
        nonlocal kp, vp, w, lens
        kn, vn = rng.standard_normal((2, B, Hkv, n, D)).astype(np.float16)
        lens = (lens + new_lens).astype(np.int32)
        kp, vp, w = OP.append(kn, vn, kp, vp, perm, lens, new_lens, w)
        gb.kv_paged_append_f16(t(kn), t(vn), gk, gv, tt, t(lens), new_lens=t(new_lens), weights=gw)

    feed(30, np.array([30, 1, 17], dtype=np.int32))
    evictions = 0
    for step in range(60):
        feed(1, np.ones(B, dtype=np.int32))
        q = (1.5 * rng.standard_normal((B, Hq, 1, D))).astype(np.float16)
        o = gb.attn_paged_decode_f16_fwd(t(q), gk, gv, tt, t(lens), weights=gw)
        ref = OP.decode(q, kp, vp, perm, lens, scale)
        e = row_error(ref["size"], D)
        assert_within(o.float().cpu().numpy(), ref["o"], 2.0 ** -11 * np.abs(ref["o"]) +
                      2.0 ** -25 + 2 * e[..., None] * ref["spread"], f"step {step}")
        w = gw.cpu().numpy()     # rank by the GPU's own weights: near ties may fall either way
        if lens.max() >= budget + ps:
            evictions += 1
            new_lens, kept = gb.kv_paged_evict(gk, gv, gw, tt, t(lens), budget, sink=2, recent=8)
            kp, vp, w, lens, rkept = OP.evict(kp, vp, w, perm, perm, lens, budget, 2, 8)
            assert np.array_equal(kept.cpu().numpy(), rkept)
            assert np.array_equal(new_lens.cpu().numpy(), lens)
        assert np.array_equal(gk.cpu().numpy().view(np.uint16), kp.view(np.uint16))
    assert evictions >= 2 and gb.device_status() == 0


def test_pages_past_32_bit_offsets(gb):
    """Pages at the end of a pool of 4.6e9 elements: append, decode with weights, eviction in place
    and into other pages give what they give in a small pool, bit for bit."""
    B, Hq, Hkv, D, ps, n_pages = 2, 8, 8, 128, 64, 24
    big = 2 ** 32 // (ps * Hkv * D) + 1 + 2 * n_pages
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(B, Hq, Hkv, 1, (700, 333), D, 41, page_size=ps,
                                                        spare_pages=7)
    P = kp.shape[0]
    assert P == n_pages and (big - P) * ps * Hkv * D > 2 ** 32
    spare = np.setdiff1d(np.arange(P), table)[:6].reshape(2, 3).astype(np.int32)
    kn, vn = np.random.default_rng(42).standard_normal((2, B, Hkv, 3, D)).astype(np.float16)

    def run(pool, first):
        gk, gv = (torch.empty((pool, ps, Hkv, D), dtype=torch.float16, device=DEV) for _ in range(2))
        gw = torch.empty((pool, Hkv, ps), device=DEV)
        mine = slice(first, first + P)
        gk[mine], gv[mine], gw[mine] = t(kp), t(vp), t(w)
        gt = t(np.where(table < 0, table, table + first).astype(np.int32))
        gl = t(lens)
        gb.kv_paged_append_f16(t(kn), t(vn), gk, gv, gt, gl, weights=gw)
        o = gb.attn_paged_decode_f16_fwd(t(q), gk, gv, gt, gl, weights=gw)
        moved = gb.kv_paged_evict(gk, gv, gw, gt, gl, 150, sink=4, recent=20, dst_table=t(spare + first))
        there = gb.kv_paged_evict(gk, gv, gw, gt, gl, 200, sink=4, recent=20)
        assert gb.device_status() == 0
        return [o, *moved, *there, gk[mine].clone(), gv[mine].clone(), gw[mine].clone()]

    small, large = run(P, 0), run(big, big - P)
    for a, b in zip(small, large):
        assert torch.equal(a, b)


def test_decodes_at_the_same_time(gb):
    """Two calls on two streams, each with a workspace of its own."""
    cases = [inputs.paged_f16_inputs(3, 8, 2, 1, (9000, 5000, 12000), 128, seed) for seed in (43, 44)]
    on_gpu = [[t(x) for x in case] for case in cases]
    want = []
    for q, kp, vp, table, lens, w in on_gpu:
        gw = w.clone()
        want.append((gb.attn_paged_decode_f16_fwd(q, kp, vp, table, lens, weights=gw), gw))
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(c[0]) for _ in range(8)] for c in on_gpu]
    sums = [[c[5].clone() for _ in range(8)] for c in on_gpu]
    ws = [torch.empty(gb.attn_paged_decode_f16_workspace_size(3, 8, 2, 1, c[3].shape[1] * 32, 128, True),
                      dtype=torch.uint8, device=DEV) for c in on_gpu]
    torch.cuda.synchronize()
    for k in range(8):
        for s, (q, kp, vp, table, lens, _), o, gw, space in zip(streams, on_gpu, outs, sums, ws):
            gb.attn_paged_decode_f16_fwd(q, kp, vp, table, lens, o=o[k], weights=gw[k],
                                         workspace=space, stream=s)
    torch.cuda.synchronize()
    for (o, gw), os, gws in zip(want, outs, sums):
        assert all(torch.equal(o, x) for x in os) and all(torch.equal(gw, x) for x in gws)


def test_shared_prefix_pages_are_evicted_into_fresh_ones(gb):
    """Two sequences over the same first pages keep different tokens of them; the shared pages and
    their weights stay as they are."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 4, 2, 1, (300, 300), 64, 45, page_size=16,
                                                        spare_pages=12)
    spare = np.setdiff1d(np.arange(kp.shape[0]), table)[:12].reshape(2, 6).astype(np.int32)
    table[1, :10] = table[0, :10]
    lens[1] = 250
    gk, gv, gw = t(kp), t(vp), t(w)
    new_lens, kept = gb.kv_paged_evict(gk, gv, gw, t(table), t(lens), 90, sink=3, recent=30,
                                       dst_table=t(spare))
    rk, rv, rw, rlens, rkept = OP.evict(kp, vp, w, table, spare, lens, 90, 3, 30)
    assert gb.device_status() == 0
    assert np.array_equal(kept.cpu().numpy(), rkept) and np.array_equal(new_lens.cpu().numpy(), rlens)
    for got, ref in ((gk, rk), (gv, rv), (gw, rw)):
        assert np.array_equal(got.cpu().numpy(), ref)


def test_wrappers_refuse_wrong_tensors(gb):
    """A wrong type, shape, stride or device of each tensor of a call is a ValueError."""
    q, kp, vp, table, lens, w = (t(x) for x in inputs.paged_f16_inputs(2, 4, 2, 1, (40, 70), 64, 46))
    k_new = torch.zeros((2, 2, 1, 64), dtype=torch.float16, device=DEV)
    calls = [(gb.kv_paged_append_f16, (k_new, k_new, kp, vp, table, lens, lens, w)),
             (gb.attn_paged_decode_f16_fwd, (q, kp, vp, table, lens, None, torch.empty_like(q), None, w)),
             (gb.kv_paged_evict, (kp, vp, w, table, lens, 16, 0, 0, table.clone()))]
    for call, args in calls:
        for i, x in enumerate(args):
            if not isinstance(x, torch.Tensor):
                continue
            wider = x.double() if x.is_floating_point() else x.long()
            for wrong in (x.cpu(), wider, x[..., :-1], x[:1].clone(), x[None]):
                with pytest.raises(ValueError):
                    call(*args[:i], wrong, *args[i + 1:])
    assert gb.device_status() == 0
