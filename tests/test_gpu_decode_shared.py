"""Decode behind shared prefixes on the GPU against the float64 decode of the same tables: the bounds are
the ordinary decode's (test_gpu_paged_f16: scores, exponentials, P in two halves, the output's
rounding), since the prefix's tokens go through the same steps."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP
from tests.test_gpu_paged_f16 import assert_within, row_error, t

pytestmark = pytest.mark.gpu
DEV = "cuda"


def shared_inputs(groups, own, Hq, Hkv, nq, D, page, seed, q_std=1.0, poison=True):
    """groups: [(sequences, prefix)]; own: tokens of each sequence behind it.  Returns (q, k_pages, v_pages,
    table as the call gets it, whole table, lens, starts, prefix_lens); rows of sequences that do not
    lead a group hold -1 in the prefix's place.  poison: NaN in every row that nobody holds."""
    rng = np.random.default_rng(seed)
    B = sum(m for m, _ in groups)
    assert len(own) == B
    prefix = [p for m, p in groups for _ in range(m)]
    own_pages = [-(-n // page) for n in own]
    P = sum(own_pages) + sum(p // page for _, p in groups) + 2
    order = rng.permutation(P).astype(np.int32)
    width = max(1, max(p // page + c for p, c in zip(prefix, own_pages))) + 1
    whole = np.full((B, width), -1, dtype=np.int32)
    call = whole.copy()
    at, b, starts = 0, 0, [0]
    for m, p in groups:
        pages = order[at:at + p // page]
        at += p // page
        for i in range(m):
            whole[b, :p // page] = pages
            if i == 0:
                call[b, :p // page] = pages
            mine = order[at:at + own_pages[b]]
            at += own_pages[b]
            for tab in (whole, call):
                tab[b, p // page:p // page + own_pages[b]] = mine
            b += 1
        starts.append(b)
    q = (rng.standard_normal((B, Hq, nq, D)) * q_std).astype(np.float16)
    kp, vp = rng.standard_normal((2, P, page, Hkv, D)).astype(np.float16)
    lens = np.array([p + n for p, n in zip(prefix, own)], dtype=np.int32)
    if poison:
        held = np.zeros((P, page), dtype=bool)
        for b in range(B):
            s = np.arange(lens[b])
            held[whole[b, s // page], s % page] = True
        kp[~held] = np.nan
        vp[~held] = np.nan
    return (q, kp, vp, call, whole, lens, np.array(starts, dtype=np.int32),
            np.array([p for _, p in groups], dtype=np.int32))


WIDE = 4096    # columns of a table whose bounds keep the call from its form for short caches


def widen(table):
    return np.concatenate([table, np.full((table.shape[0], WIDE), -1, dtype=np.int32)], 1)


def check(gb, groups, own, Hq, Hkv, nq, D, page, seed=1, q_std=1.0, workspace=None, bounds=True, x=None):
    """The call against the oracle, with bounds that let short caches take their form (one kernel) and with
    a wide table that does not (two).  Returns the latter's (o, lse)."""
    x = x or shared_inputs(groups, own, Hq, Hkv, nq, D, page, seed, q_std)
    for wide in (False, True):
        q, kp, vp, call, whole, lens, starts, pre = x
        scale = inputs.softmax_scale(D)
        lse = torch.full(q.shape[:3], 7.0, device=DEV)
        kw = dict(max_prefix_len=int(pre.max()), max_own_len=max(own)) if bounds and not wide else {}
        table = widen(call) if wide else call
        if workspace:
            most = table.shape[1] * page
            size = gb.attn_paged_decode_shared_f16_workspace_size(
                q.shape[0], Hq, Hkv, nq, len(pre), kw.get("max_prefix_len", most),
                kw.get("max_own_len", most), D)
            kw["workspace"] = torch.empty(int(size * workspace), dtype=torch.uint8, device=DEV)
        before = gb.launch_count()
        o = gb.attn_paged_decode_shared_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), t(starts), t(pre),
                                                lse=lse, scale=scale, **kw)
        assert gb.device_status() == 0 and (not wide or gb.launch_count() == before + 2)
        ref = OP.decode(q, kp, vp, whole, lens, scale)
        e = row_error(ref["size"], D)
        assert_within(o.float().cpu().numpy(), ref["o"],
                      2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], "o")
        with np.errstate(invalid="ignore"):
            assert_within(lse.cpu().numpy(), ref["lse"], e + 2.0 ** -23 * np.abs(ref["lse"]), "lse")
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_group(gb, D, page):
    check(gb, [(5, 512)], [1, 17, 300, 64, 2], 8, 2, 1, D, page)
    check(gb, [(3, 256)], [40, 0, 1], 6, 1, 1, D, page, seed=2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefix_lengths_around_the_tiles(gb, D):
    for prefix in (16, 48, 64, 80, 112, 128, 144, 1040):
        check(gb, [(2, prefix)], [5, 33], 4, 2, 1, D, 16, seed=prefix)


@pytest.mark.parametrize("D,Hq,Hkv,nq", [(128, 32, 8, 1), (256, 6, 1, 2), (64, 12, 3, 1), (128, 16, 1, 3),
                                         (256, 32, 2, 1), (64, 40, 1, 4), (128, 5, 5, 2)])
def test_several_groups(gb, D, Hq, Hkv, nq):
    """Groups of many sequences, of one, of none; with and without a prefix; more rows than a unit."""
    check(gb, [(9, 320), (1, 0), (0, 64), (1, 1600), (4, 16), (3, 0), (0, 0), (2, 704)],
          [1, 100, 33, 64, 7, 0, 250, 16, 15, 77, 9, 300, 40, 41, 42, 1, 2, 500, 128, 90], Hq, Hkv, nq, D, 16,
          seed=D + nq)


def test_rows_around_a_unit(gb):
    for B, Hq, Hkv, nq in ((31, 4, 1, 1), (32, 4, 1, 1), (33, 4, 1, 1), (43, 6, 2, 2), (128, 3, 1, 1),
                           (1, 130, 1, 1), (2, 200, 1, 2)):
        check(gb, [(B, 192)], [(7 * i) % 40 for i in range(B)], Hq, Hkv, nq, 128, 16, seed=B)


def test_queries_within_the_prefix(gb):
    """More queries than own tokens: the first of them sit in the prefix, or before its first token."""
    check(gb, [(3, 128), (2, 16), (1, 0)], [0, 2, 4, 1, 0, 3], 4, 2, 5, 128, 16)
    check(gb, [(3, 16), (1, 32)], [0, 1, 5, 3], 2, 1, 20, 256, 16, seed=2)
    check(gb, [(2, 64)], [0, 0], 2, 1, 130, 64, 32, seed=3)


def test_no_tokens_at_all(gb):
    o, lse = check(gb, [(2, 0), (1, 0)], [0, 0, 0], 4, 2, 1, 128, 16)
    assert not o.any() and torch.isneginf(lse).all()
    check(gb, [(3, 64)], [0, 0, 0], 4, 2, 1, 128, 16)              # nothing but the prefix
    check(gb, [(3, 0)], [5, 600, 0], 4, 2, 1, 128, 16)             # nothing in common


def test_defaults_and_wide_scores(gb):
    check(gb, [(6, 320)], [30, 1, 0, 64, 100, 9], 8, 2, 1, 128, 64, bounds=False)
    check(gb, [(6, 640)], [30, 1, 0, 64, 100, 9], 8, 2, 1, 128, 64, q_std=12.0, seed=4)
    check(gb, [(4, 640)], [300, 11, 7, 64], 6, 1, 2, 256, 32, q_std=12.0, seed=5)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prefixes_over_all_ctas(gb, D):
    check(gb, [(20, 8192)], [(37 * i) % 400 for i in range(20)], 8, 2, 1, D, 64, seed=6)
    check(gb, [(1, 12000), (2, 4000)], [700, 2500, 3], 4, 1, 1, D, 32, seed=7)


def test_many_groups(gb):
    rng = np.random.default_rng(8)
    groups = [(int(rng.integers(0, 4)), 16 * int(rng.integers(0, 12))) for _ in range(300)]
    own = [int(rng.integers(0, 60)) for _ in range(sum(m for m, _ in groups))]
    check(gb, groups, own, 2, 1, 1, 64, 16)
    check(gb, [(1, 16)] * 700, [i % 3 for i in range(700)], 2, 2, 1, 128, 16, seed=9)


def test_4096_sequences(gb):
    check(gb, [(4000, 64), (96, 32)], [i % 18 for i in range(4096)], 2, 1, 1, 64, 16, seed=10)


def test_small_workspaces(gb):
    """Fewer CTAs, the same result within the bounds; too few is refused."""
    for part in (0.9, 0.5):
        check(gb, [(6, 2048)], [300, 1, 0, 64, 100, 9], 8, 2, 1, 128, 64, workspace=part)
    with pytest.raises(gb.GbattnError) as e:
        check(gb, [(6, 2048)], [300, 1, 0, 64, 100, 9], 8, 2, 1, 128, 64, workspace=0.01)
    assert e.value.status == 6


@pytest.mark.parametrize("wide", [False, True])
def test_equals_the_ordinary_decode(gb, wide):
    """The same tables through both calls."""
    x = shared_inputs([(7, 960), (2, 0)], [30, 1, 0, 64, 100, 9, 200, 5, 3000], 16, 4, 1, 128, 16, 11)
    q, kp, vp, _, whole, lens, starts, pre = x
    a = gb.attn_paged_decode_shared_f16_fwd(t(q), t(kp), t(vp), t(widen(whole) if wide else whole), t(lens), t(starts), t(pre))
    b = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(whole), t(lens))
    assert gb.device_status() == 0
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -10 * b.float().abs().max()


@pytest.mark.parametrize("wide", [False, True])
def test_infinite_values_stay_in_their_group(gb, wide):
    groups, own = [(3, 320), (2, 64)], [20, 1, 40, 30, 9]
    x = shared_inputs(groups, own, 4, 2, 1, 128, 16, 12)
    q, kp, vp, call, whole, lens, starts, pre = x
    args = [t(a) for a in (q, kp, vp, widen(call) if wide else call, lens, starts, pre)]
    clean = gb.attn_paged_decode_shared_f16_fwd(*args)
    vp = vp.copy()
    vp[whole[0, 19], 3, 1, 5] = np.inf                  # in the first group's prefix, KV head 1
    args[2] = t(vp)
    o = gb.attn_paged_decode_shared_f16_fwd(*args)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[:3, 2:, :, 5] = True
    assert torch.equal(o[~bad], clean[~bad]) and not torch.isfinite(o[bad]).any()
    assert gb.device_status() == 0


def rejected(gb, x, good, flag, launches, **kw):
    """The sequences of `good` come out as without the others' faults, the rest as O = 0."""
    q, kp, vp, call, whole, lens, starts, pre = x
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    before = gb.launch_count()
    o = gb.attn_paged_decode_shared_f16_fwd(t(q), t(kp), t(vp), t(call), t(lens), t(starts), t(pre), lse=lse,
                                            **kw)
    assert gb.launch_count() - before == launches and gb.device_status() == flag
    o, lse = o.float().cpu().numpy(), lse.cpu().numpy()
    bad = np.setdiff1d(np.arange(q.shape[0]), good)
    assert not o[bad].any() and np.isneginf(lse[bad]).all()
    if len(good):
        ref = OP.decode(q[good], kp, vp, whole[good], lens[good], inputs.softmax_scale(q.shape[3]))
        e = row_error(ref["size"], q.shape[3])
        assert_within(o[good], ref["o"],
                      2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], "o")


# KV heads of six sequences: streams for the form for short caches, and too many of them for it
FORMS = pytest.mark.parametrize("Hkv,launches", [(2, 1), (40, 2)])


@FORMS
def test_bad_lengths(gb, Hkv, launches):
    groups, own = [(2, 64), (3, 128), (1, 0)], [10, 20, 30, 40, 50, 60]

    def fresh():
        return list(shared_inputs(groups, own, 2 * Hkv, Hkv, 1, 128, 16, 13))
    x = fresh()
    x[5] = x[5].copy()
    x[5][1], x[5][2], x[5][5] = 63, 128 + 61, -1       # below the prefix, above max_own_len, negative
    rejected(gb, x, [0, 3, 4], gb.DEV_BAD_LENGTH, launches, max_own_len=60, max_prefix_len=128)
    x = fresh()                                        # a length past the table's row
    x[5] = x[5].copy()
    cap = 16 * x[3].shape[1]                           # (its own part alone would fit)
    x[5][5], x[5][4], x[5][3] = cap + 1, 2 ** 31 - 1, cap + 10
    rejected(gb, x, [0, 1, 2], gb.DEV_BAD_LENGTH, launches)
    for bad in (-16, 136, 144, 2 ** 31 - 1):           # a prefix that is none
        x = fresh()
        x[7] = x[7].copy()
        x[7][1] = bad
        rejected(gb, x, [0, 1, 5], gb.DEV_BAD_LENGTH, launches, max_own_len=60, max_prefix_len=128)
    for starts in ([0, 2, 5, 7], [0, 2, 5, 5], [1, 2, 5, 6], [0, 5, 2, 6], [0, -3, 5, 6],
                   [0, 2 ** 31 - 1, 5, 6], [-2 ** 31, 2, 5, 6]):
        x = fresh()
        x[6] = np.array(starts, dtype=np.int32)
        rejected(gb, x, [], gb.DEV_BAD_INDEX, launches)


def test_bad_lengths_among_many_sequences(gb):
    """As above where the merge reads the tables that the decode kernel left (more than 64 sequences)."""
    x = list(shared_inputs([(60, 64), (20, 32), (5, 0)], [3 + i % 30 for i in range(85)], 4, 2, 1, 64, 16, 21))
    x[5] = x[5].copy()
    x[5][7], x[5][70], x[5][84] = 63, 16 * x[3].shape[1] + 5, -9
    good = np.setdiff1d(np.arange(85), [7, 70, 84])
    rejected(gb, x, good, gb.DEV_BAD_LENGTH, 2)
    x[7] = np.array([64, 33, 0], dtype=np.int32)
    rejected(gb, x, np.setdiff1d(good, np.arange(60, 80)), gb.DEV_BAD_LENGTH, 2)
    x[6] = np.array([0, 60, 59, 85], dtype=np.int32)
    rejected(gb, x, [], gb.DEV_BAD_INDEX | gb.DEV_BAD_LENGTH, 2)


@pytest.mark.parametrize("wide", [False, True])
def test_bad_pages(gb, wide):
    """An entry that is none is reported; the other group is not touched by it."""
    x = list(shared_inputs([(2, 128), (2, 64)], [10, 20, 30, 40], 4, 2, 1, 128, 16, 14, poison=False))
    q, kp, vp, call, whole, lens, starts, pre = x
    call[0, 3], call[2, 4] = kp.shape[0], -7           # a prefix page, an own page
    call = widen(call) if wide else call
    o = gb.attn_paged_decode_shared_f16_fwd(t(q), t(kp), t(vp), t(call), t(lens), t(starts), t(pre))
    assert gb.device_status() == gb.DEV_BAD_PAGE
    ref = OP.decode(q[3:], kp, vp, whole[3:], lens[3:], inputs.softmax_scale(128))
    assert np.abs(o[3:].float().cpu().numpy() - ref["o"]).max() < 2e-3


@pytest.mark.parametrize("wide", [False, True])
def test_pool_past_32_bit_offsets(gb, wide):
    page, Hkv, D, P = 64, 8, 256, 20000                # 2.6 GB a tensor's elements pass 2^31
    kp = torch.zeros((P, page, Hkv, D), dtype=torch.float16, device=DEV)
    vp = torch.zeros_like(kp)
    rng = np.random.default_rng(15)
    used = np.array([P - 1, 17000, P - 2, 5])
    k, v = rng.standard_normal((2, 4, page, Hkv, D)).astype(np.float16)
    kp[torch.from_numpy(used).to(DEV)], vp[torch.from_numpy(used).to(DEV)] = t(k), t(v)
    q = rng.standard_normal((2, 8, 1, D)).astype(np.float16)
    lens = np.array([140, 192], dtype=np.int32)
    table = np.array([[0, 1, 2], [0, 1, 3]], dtype=np.int32)
    o = gb.attn_paged_decode_shared_f16_fwd(t(q), kp, vp, t(widen(used[table].astype(np.int32)) if wide else
                                                      used[table].astype(np.int32)), t(lens),
                                            t(np.array([0, 2], dtype=np.int32)),
                                            t(np.array([128], dtype=np.int32)))
    assert gb.device_status() == 0
    ref = OP.decode(q, k, v, table, lens, inputs.softmax_scale(D))
    assert_within(o.float().cpu().numpy(), ref["o"], 2e-3 + 1e-2 * np.abs(ref["o"]), "o")


@pytest.mark.parametrize("wide", [False, True])
def test_graph_side_stream_and_repeats(gb, wide):
    """Replays of a captured call, and a call on a side stream, give the eager call's bits."""
    x = shared_inputs([(6, 1024), (3, 320)], [30, 1, 0, 64, 100, 9, 200, 5, 300], 8, 2, 1, 128, 16, 16)
    args = [t(x[i]) for i in (0, 1, 2, 3, 5, 6, 7)]
    kw = dict(max_prefix_len=1024, max_own_len=300)
    if wide:
        args[3] = t(widen(x[3]))
        kw = dict(max_prefix_len=1024, max_own_len=30000)
    want = gb.attn_paged_decode_shared_f16_fwd(*args, **kw)
    size = gb.attn_paged_decode_shared_f16_workspace_size(9, 8, 2, 1, 2, 1024, kw["max_own_len"], 128)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)       # NaN everywhere
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gb.attn_paged_decode_shared_f16_fwd(*args, o=out, workspace=ws, **kw)
    for _ in range(20):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    got = gb.attn_paged_decode_shared_f16_fwd(*args, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got, want) and gb.device_status() == 0


@pytest.mark.parametrize("mode", [1, 2])
def test_waits_that_run_out_in_clusters(gb, mode):
    x = shared_inputs([(4, 2048)], [1000, 3, 200, 64], 8, 1, 1, 128, 64, 18)
    args = [t(x[i]) for i in (0, 1, 2, 3, 5, 6, 7)]
    kw = dict(max_prefix_len=2048, max_own_len=1000)
    before = gb.launch_count()
    want = gb.attn_paged_decode_shared_f16_fwd(*args, **kw)
    assert gb.device_status() == 0 and gb.launch_count() == before + 1
    gb.set_wait_limit_ns(20_000_000)
    gb.test_inject_fault(mode)
    try:
        gb.attn_paged_decode_shared_f16_fwd(*args, **kw)
        assert gb.device_status() in (gb.DEV_WAIT_TIMEOUT, 0 if mode == 2 else gb.DEV_WAIT_TIMEOUT)
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(gb.attn_paged_decode_shared_f16_fwd(*args, **kw), want) and gb.device_status() == 0


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("D", [128, 256])
def test_waits_that_run_out(gb, mode, D):
    """Nothing is loaded, or loading stops in mid-stream: the call ends by itself and says so."""
    x = shared_inputs([(40, 65536)], [(37 * i) % 900 for i in range(40)], 8, 1, 1, D, 64, 17)
    args = [t(x[i]) for i in (0, 1, 2, 3, 5, 6, 7)]
    want = gb.attn_paged_decode_shared_f16_fwd(*args)
    assert gb.device_status() == 0
    gb.set_wait_limit_ns(20_000_000)
    gb.test_inject_fault(mode)
    try:
        gb.attn_paged_decode_shared_f16_fwd(*args)
        assert gb.device_status() == gb.DEV_WAIT_TIMEOUT
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(gb.attn_paged_decode_shared_f16_fwd(*args), want) and gb.device_status() == 0
