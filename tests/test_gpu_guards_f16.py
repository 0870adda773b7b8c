"""Guard bands around every output of the calls on paged FP16 caches and of differential attention:
ragged sizes write nothing outside o, lse, new_lens, kept, the pool's slots and the weights."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import diff as OD
from oracle import paged as OP
from test_gpu_guards import Guarded, close, t

pytestmark = pytest.mark.gpu


def guarded(x):
    """A guarded copy of an array."""
    g = Guarded(x.shape, torch.from_numpy(x).dtype)
    g.view.copy_(t(x))
    return g


@pytest.mark.parametrize("bound", [None, 100000])   # in clusters, and as a chain with a merge
@pytest.mark.parametrize("D,Hq,nq", [(64, 3, 1), (128, 20, 1), (256, 5, 3), (128, 9, 2)])
def test_guards_decode_f16(gb, D, Hq, nq, bound):
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, Hq, 1, nq, (333, 0, 17), D, 121, page_size=16)
    if bound is not None:
        wide = np.full((3, bound // 16), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
    else:
        wide = table
    o, lse = Guarded(q.shape, torch.float16), Guarded(q.shape[:3], torch.float32)
    gw, k, v = guarded(w), guarded(kp), guarded(vp)
    gb.attn_paged_decode_f16_fwd(t(q), k.view, v.view, t(wide), t(lens), o=o.view, lse=lse.view,
                                 weights=gw.view)
    assert gb.device_status() == 0
    ref = OP.decode(q, kp, vp, table, lens, inputs.softmax_scale(D))
    assert all(g.intact() for g in (o, lse, gw, k, v))
    assert close(o.view.float().cpu().numpy(), ref["o"])
    held = np.zeros(w.shape, dtype=bool)
    for b, n in enumerate(lens):
        held[table[b, np.arange(n) // 16], :, np.arange(n) % 16] = True
    assert np.array_equal(gw.view.cpu().numpy()[~held], w[~held])


@pytest.mark.parametrize("bound", [None, 100000])
@pytest.mark.parametrize("Hq,nq", [(3, 1), (20, 1), (5, 3)])
def test_guards_diff_decode(gb, Hq, nq, bound):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(3, Hq, 1, nq, (333, 0, 17), 128, 122, page_size=16)
    wide = np.full((3, table.shape[1] if bound is None else bound // 16), -1, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    vecs, weight = inputs.diff_inputs(Hq, 128, 123)
    o, lse = Guarded(q.shape, torch.float16), Guarded((3, Hq, 2, nq), torch.float32)
    gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(wide), t(lens), t(vecs), 0.5,
                                      norm_weight=t(weight), o=o.view, lse=lse.view)
    assert gb.device_status() == 0 and o.intact() and lse.intact()
    ref = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.5, 0.125, weight)
    assert close(o.view.float().cpu().numpy(), ref["o"])


@pytest.mark.parametrize("Sq,Skv", [(70, 90), (200, 133), (130, 5000)])   # the last in split key ranges
def test_guards_diff_prompt(gb, Sq, Skv):
    rng = np.random.default_rng(124)
    q, k, v = (rng.standard_normal((2, h, n, 128)).astype(np.float16) for h, n in
               ((4, Sq), (2, Skv), (2, Skv)))
    ql, kl = np.array([Sq, Sq // 2], np.int32), np.array([Skv, Skv - 7], np.int32)
    vecs, weight = inputs.diff_inputs(4, 128, 125)
    o, lse = Guarded(q.shape, torch.float16), Guarded((2, 4, 2, Sq), torch.float32)
    n = gb.attn_diff_prefill_workspace_size(2, 4, Sq, Skv, 128)
    assert (n > 0) == (Skv == 5000)
    ws = Guarded((max(n // 4, 4),), torch.int32)
    gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.5, norm_weight=t(weight), q_lens=t(ql),
                             kv_lens=t(kl), o=o.view, lse=lse.view, workspace=ws.view)
    assert gb.device_status() == 0 and o.intact() and lse.intact() and ws.intact()
    ref = OD.prefill(q, k, v, vecs, 0.5, 0.125, weight, q_lens=ql, kv_lens=kl)
    got = o.view.float().cpu().numpy()
    assert close(got, ref["o"]) and np.all(got[1, :, Sq // 2:] == 0)


@pytest.mark.parametrize("D,elem", [(64, 2), (256, 2), (64, 1)])
@pytest.mark.parametrize("in_place", [True, False])
def test_guards_append_and_evict(gb, D, elem, in_place):
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(3, 3, 3, 1, (333, 20, 64), D, 126, page_size=16,
                                                        spare_pages=15)
    spare = np.setdiff1d(np.arange(kp.shape[0]), table[table >= 0])[:15].reshape(3, 5).astype(np.int32)
    rng = np.random.default_rng(127)
    if elem == 2:
        kn, vn = rng.standard_normal((2, 3, 3, 5, D)).astype(np.float16)
        k, v, gw = guarded(kp), guarded(vp), guarded(w)
        gb.kv_paged_append_f16(t(kn), t(vn), k.view, v.view, t(table), t(lens), weights=gw.view)
        assert gb.device_status() == 0 and k.intact() and v.intact() and gw.intact()
        kp, vp, w = OP.append(kn, vn, kp, vp, table, lens, None, w)
        assert np.array_equal(k.view.cpu().numpy(), kp) and np.array_equal(gw.view.cpu().numpy(), w)
    else:
        kp, vp = (x.view(np.uint8)[..., ::2].copy() for x in (kp, vp))
        k, v, gw = t(kp), t(vp), guarded(w)
    new_lens, kept = Guarded((3,), torch.int32), Guarded((3, 3, 75), torch.int32)
    pools = [x.view if elem == 2 else x for x in (k, v)]
    gb.kv_paged_evict(*pools, gw.view, t(table), t(lens), 75, sink=3, recent=20,
                      dst_table=None if in_place else t(spare), new_lens=new_lens.view, kept=kept.view)
    assert gb.device_status() == 0
    dst = table if in_place else spare
    rk, rv, rw, rl, rkept = OP.evict(kp, vp, w, table, dst, lens, 75, 3, 20)
    assert all(g.intact() for g in (new_lens, kept, gw)) and (elem == 1 or (k.intact() and v.intact()))
    assert np.array_equal(new_lens.view.cpu().numpy(), rl) and np.array_equal(kept.view.cpu().numpy(), rkept)
    for got, ref in zip(pools, (rk, rv)):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert np.array_equal(gw.view.cpu().numpy(), rw)
