"""The FP16 decodes of short caches (one kernel in clusters) when loading stops in the middle of a warp's
tiles: the wait runs out, the call ends by itself and says so, and the next one is right."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from tests.test_gpu_decode_shared import shared_inputs, t

pytestmark = pytest.mark.gpu
DEV = "cuda"


def stops_and_recovers(gb, call):
    before = gb.launch_count()
    want = call().clone()
    assert gb.device_status() == 0 and gb.launch_count() == before + 1      # the form in clusters
    gb.set_wait_limit_ns(20_000_000)
    gb.test_inject_fault(2)
    try:
        call()
        assert gb.device_status() == gb.DEV_WAIT_TIMEOUT
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(call(), want) and gb.device_status() == 0


# At D = 256 the form is taken with one tile a warp at most: there is no middle to stop in.
@pytest.mark.parametrize("D", [64, 128])
def test_loads_that_stop_behind_a_prefix(gb, D):
    x = shared_inputs([(4, 2048)], [1000, 3, 200, 64], 8, 1, 1, D, 64, 18)
    args = [t(x[i]) for i in (0, 1, 2, 3, 5, 6, 7)]
    stops_and_recovers(gb, lambda: gb.attn_paged_decode_shared_f16_fwd(*args, max_prefix_len=2048, max_own_len=1000))


@pytest.mark.parametrize("D", [64, 128])
def test_loads_that_stop(gb, D):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(4, 8, 1, 1, (3048, 2051, 2248, 2112), D, 19)
    args = [t(x) for x in (q, kp, vp, table, lens)]
    stops_and_recovers(gb, lambda: gb.attn_paged_decode_f16_fwd(*args, max_kv_len=3048))
