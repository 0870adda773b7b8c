"""The FP16 decodes as a chain of kernels (tiles laid end to end, partial records, merge, weights):
lengths or a length bound above what the one-kernel form takes.  Bounds as in the tests of the calls."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import diff as OD
from test_gpu_diff import assert_diff
from test_gpu_paged_f16 import check_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def widened(table, ps, bound):
    """The same table for a bound of `bound` tokens a sequence, -1 past the pages in use."""
    wide = np.full((table.shape[0], bound // ps), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    return wide


def check_diff(gb, B, Hq, Hkv, nq, lens, bound, seed, norm=True, heads=None, workspace=None, ps=16,
               kernels=2):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(B, Hq, Hkv, nq, lens, D, seed, page_size=ps,
                                                        spare_pages=1, poison=True)
    vecs, weight = inputs.diff_inputs(Hq, D, seed + 1, heads=heads, norm=norm)
    lse = torch.full((B, Hq, 2, nq), 7.0, device=DEV)
    before = gb.launch_count()
    o = gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(widened(table, ps, bound)), t(lens),
                                          t(vecs), 0.55, norm_weight=t(weight), lse=lse,
                                          workspace=workspace)
    assert gb.device_status() == 0 and gb.launch_count() - before == kernels
    ref = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.55, 0.125, weight)
    assert_diff(o, lse, ref, weight, 0.55, 2.0 ** -22)


@pytest.mark.parametrize("Hq,Hkv,nq", [(1, 1, 1), (4, 1, 1), (8, 2, 1), (5, 1, 1), (6, 2, 3),
                                       (16, 1, 1), (9, 1, 2), (24, 1, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_decode_merged(gb, Hq, Hkv, nq, norm):
    """Rows below, at and above one row group; lengths down to one and none."""
    check_diff(gb, 4, Hq, Hkv, nq, (700, 1, 0, 65), 100000, 101, norm=norm)


@pytest.mark.parametrize("Hq,nq", [(16, 1), (32, 1), (16, 2), (64, 1), (24, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_decode_row_groups_side_by_side(gb, Hq, nq, norm):
    """A bound above 256 MB of cache: 2, 4 and 8 row groups share a CTA's tiles, three do not."""
    check_diff(gb, 3, Hq, 1, nq, (1300, 0, 70), 400000, 103, norm=norm)


@pytest.mark.parametrize("B", [64, 65, 300])
def test_diff_decode_many_sequences(gb, B):
    """Tile counts summed from the lengths up to 64 sequences, read from the decode's table above."""
    lens = tuple(int(x) for x in np.random.default_rng(B).integers(0, 90, B))
    check_diff(gb, B, 4, 1, 2, lens, 100000, 105, heads=1)


def test_diff_decode_merged_with_less_workspace(gb):
    """Down to one CTA's worth: eight long warp ranges that cut several sequences each."""
    full = gb.attn_diff_paged_decode_f16_workspace_size(3, 4, 2, 1, 100000, D)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    record = 8 * (D * 4 + 8)
    for ctas in (sms - 1, 40, 3, 1):
        ws = torch.full((full - (sms - ctas) * record,), 0xFF, dtype=torch.uint8, device=DEV)
        check_diff(gb, 3, 4, 2, 1, (2500, 3, 900), 100000, 107, workspace=ws)


def test_decode_long_caches_with_less_workspace(gb):
    """Lengths past the clusters' limit; the workspace's contents do not matter, one CTA's worth is
    enough, less is refused, and two calls give the same bits."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 8, 2, 1, (7000, 6500), D, 109)
    bound = table.shape[1] * 32
    assert bound > 6144
    full = gb.attn_paged_decode_f16_workspace_size(2, 8, 2, 1, bound, D, True)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    record = 8 * (D * 4 + 8)
    for ctas in (sms, 20, 1):
        ws = torch.full((full - (sms - ctas) * record,), 0xFF, dtype=torch.uint8, device=DEV)
        before = gb.launch_count()
        a, wa = check_decode(gb, q, kp, vp, table, lens, w, workspace=ws)
        assert gb.launch_count() - before == 3
        b, wb = check_decode(gb, q, kp, vp, table, lens, w, workspace=ws)
        assert torch.equal(a, b) and np.array_equal(wa, wb)
    with pytest.raises(gb.GbattnError):
        check_decode(gb, q, kp, vp, table, lens, w, workspace=torch.empty(
            full - sms * record, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("call", ["decode", "weights", "diff"])
def test_the_chain_in_a_graph_and_on_a_side_stream(gb, call):
    """Captured with its dependent launches, then replayed on other lengths, queries and weights."""
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, 8, 2, 1, (9000, 8000, 7000), D, 111)
    tq, tk, tv, tt, tl, tw = (t(x) for x in (q, kp, vp, table, lens, w))
    vecs, norm = (t(x) for x in inputs.diff_inputs(8, D, 112))
    o = torch.empty_like(tq)
    bound = table.shape[1] * 32
    n = max(gb.attn_paged_decode_f16_workspace_size(3, 8, 2, 1, bound, D, True),
            gb.attn_diff_paged_decode_f16_workspace_size(3, 8, 2, 1, bound, D))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def run(**kw):
        if call == "diff":
            return gb.attn_diff_paged_decode_f16_fwd(tq, tk, tv, tt, tl, vecs, 0.4, norm_weight=norm, **kw)
        return gb.attn_paged_decode_f16_fwd(tq, tk, tv, tt, tl, weights=tw if call == "weights" else None,
                                            **kw)

    def state():
        return [o.clone(), tw.clone()]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    before = gb.launch_count()
    with torch.cuda.graph(graph):
        run(o=o, workspace=ws)
    assert gb.launch_count() - before == (3 if call == "weights" else 2)
    for new, factor in (((9000, 8000, 7000), 1.0), ((1, 7999, 0), 0.5), ((8001, 17, 6999), 2.0)):
        tl.copy_(t(np.array(new, dtype=np.int32)))
        tq.copy_(t(q) * factor)
        results = []
        for how in ("direct", "graph", "side"):
            tw.copy_(t(w))
            torch.cuda.synchronize()
            if how == "graph":
                ws.fill_(0xFF)
                graph.replay()
            else:
                run(o=o, stream=side if how == "side" else None)
            torch.cuda.synchronize()
            results.append(state())
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    assert gb.device_status() == 0


@pytest.mark.parametrize("mode", [1, 2])   # nothing is loaded; loads stop after two rounds of a ring
@pytest.mark.parametrize("diff", [False, True])
def test_abandoned_loads_are_reported(gb, mode, diff):
    """One CTA's worth of workspace makes every warp's range longer than what mode 2 loads."""
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(2, 4, 2, 1, (9000, 450), D, 113)
    vecs, _ = inputs.diff_inputs(4, D, 114, norm=False)
    bound = table.shape[1] * 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = gb.attn_diff_paged_decode_f16_workspace_size if diff else gb.attn_paged_decode_f16_workspace_size
    full = size(2, 4, 2, 1, bound, D)
    ws = torch.empty(full - (sms - 1) * 8 * (D * 4 + 8), dtype=torch.uint8, device=DEV)
    args = [t(x) for x in (q, kp, vp, table, lens)]

    def run():
        if diff:
            return gb.attn_diff_paged_decode_f16_fwd(*args, t(vecs), 0.5, workspace=ws)
        return gb.attn_paged_decode_f16_fwd(*args, workspace=ws)
    want = run()
    assert gb.device_status() == 0
    gb.set_wait_limit_ns(20_000_000)
    try:
        gb.test_inject_fault(mode)
        run()
        assert gb.device_status() & gb.DEV_WAIT_TIMEOUT
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(run(), want) and gb.device_status() == 0
