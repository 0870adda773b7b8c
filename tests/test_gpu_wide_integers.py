"""Integers that do not fit the 32 bits that the library takes are refused, not cut to their low bits."""

import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_integers_past_32_bits(gb):
    q, kp, vp, table, lens, w = (torch.from_numpy(x).to(DEV) for x in
                                 inputs.paged_f16_inputs(2, 4, 2, 1, (40, 70), 128, 97))
    vecs = torch.zeros((4, 64), device=DEV)
    before = w.clone()
    for past in (2 ** 32, 2 ** 32 + 64, -2 ** 32 + 64, 2 ** 31):
        for call in (lambda: gb.attn_paged_decode_f16_fwd(q, kp, vp, table, lens, max_kv_len=past),
                     lambda: gb.attn_diff_paged_decode_f16_fwd(q, kp, vp, table, lens, vecs, 0.5,
                                                               max_kv_len=past),
                     lambda: gb.kv_paged_evict(kp, vp, w, table, lens, past),
                     lambda: gb.kv_paged_evict(kp, vp, w, table, lens, 16, sink=past),
                     lambda: gb.kv_paged_evict(kp, vp, w, table, lens, 16, recent=past),
                     lambda: gb.kv_paged_evict(kp, vp, w, table, lens, 16, max_kv_len=past)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    assert gb.device_status() == 0 and torch.equal(w, before)
