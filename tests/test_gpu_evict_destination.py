"""Eviction into pages that the sequence itself still needs is refused; into its own pages that the call
does not read it is not."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


# a middle to choose from; a cache within the budget; no middle, the sinks' page; the recent tokens'
@pytest.mark.parametrize("length,budget,sink,recent,same", [(200, 64, 4, 16, 1), (30000, 2000, 4, 16, 60),
                                                            (50, 64, 4, 16, 3), (200, 64, 20, 44, 1),
                                                            (70, 64, 0, 64, 3)])
def test_a_copy_of_the_page_table_is_refused(gb, length, budget, sink, recent, same):
    """Sequence 0's destination is its own page in one place (or in every); sequence 1's are fresh."""
    need = -(-budget // 16)
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 2, 2, 1, (length, 300), 64, 91, page_size=16,
                                                        spare_pages=2 * need)
    spare = np.setdiff1d(np.arange(kp.shape[0]), table)[:2 * need].reshape(2, need).astype(np.int32)
    rk, rv, rw, rl, rkept = OP.evict(kp, vp, w, table[1:], spare[1:], lens[1:], budget, sink, recent)
    one = spare.copy()
    one[0, same] = table[0, same]
    for dst in (one, np.stack([np.resize(table[0], need), spare[1]])):
        gk, gv, gw = t(kp), t(vp), t(w)
        new_lens, kept = gb.kv_paged_evict(gk, gv, gw, t(table), t(lens), budget, sink=sink,
                                           recent=recent, dst_table=t(dst))
        assert gb.device_status() == gb.DEV_BAD_PAGE
        assert new_lens.cpu().tolist() == [length, int(rl[0])]
        assert torch.all(kept[0] == -1) and np.array_equal(kept[1:].cpu().numpy(), rkept)
        for got, ref in ((gk, rk), (gv, rv), (gw, rw)):
            assert np.array_equal(got.cpu().numpy(), ref)


def test_a_window_into_the_first_pages(gb):
    """Nothing but the newest tokens is kept, and the first pages hold none of them."""
    _, kp, vp, table, lens, w = inputs.paged_f16_inputs(2, 2, 2, 1, (200, 150), 64, 92, page_size=16)
    dst = table[:, :3].copy()
    gk, gv, gw = t(kp), t(vp), t(w)
    new_lens, kept = gb.kv_paged_evict(gk, gv, gw, t(table), t(lens), 48, recent=48, dst_table=t(dst))
    assert gb.device_status() == 0
    rk, rv, rw, rl, rkept = OP.evict(kp, vp, w, table, dst, lens, 48, 0, 48)
    assert np.array_equal(new_lens.cpu().numpy(), rl) and np.array_equal(kept.cpu().numpy(), rkept)
    for got, ref in ((gk, rk), (gv, rv), (gw, rw)):
        assert np.array_equal(got.cpu().numpy(), ref)
