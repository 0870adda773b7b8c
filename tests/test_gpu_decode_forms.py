"""The FP16 decode's two forms, one kernel in clusters and a chain of two or three kernels: both right
around the stream counts where the cluster's size changes, and chosen by what they cost."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def launches(gb, B, Hkv, D, n, weights, Hq=None):
    Hq = 4 * Hkv if Hq is None else Hq
    pages = -(-n // 64)
    k = torch.zeros((B * pages, 64, Hkv, D), dtype=torch.float16, device=DEV)
    table = torch.arange(B * pages, dtype=torch.int32, device=DEV).view(B, pages)
    q = torch.zeros((B, Hq, 1, D), dtype=torch.float16, device=DEV)
    w = torch.zeros((B * pages, Hkv, 64), device=DEV) if weights else None
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    before = gb.launch_count()
    gb.attn_paged_decode_f16_fwd(q, k, k.clone(), table, lens, max_kv_len=n, weights=w)
    return gb.launch_count() - before


@pytest.mark.parametrize("B,Hkv,D,n,weights,kernels", [
    (1, 8, 128, 4096, False, 1), (1, 8, 128, 8192, False, 2), (1, 8, 128, 2048, True, 1),
    (1, 8, 128, 4096, True, 3), (12, 1, 128, 6144, True, 1), (1, 1, 64, 8192, False, 1),
    (1, 1, 64, 12288, False, 2), (8, 1, 64, 12288, False, 1), (1, 1, 256, 512, False, 2),
    (8, 1, 256, 512, False, 1), (1, 1, 256, 512, True, 1), (152, 1, 128, 768, False, 1),
    (153, 1, 128, 64, False, 2)])
def test_the_form_that_costs_less(gb, B, Hkv, D, n, weights, kernels):
    assert launches(gb, B, Hkv, D, n, weights) == kernels


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("streams", [14, 15, 16, 19, 20, 36, 37, 38, 76, 77, 151, 152, 153])
def test_around_the_clusters_that_run_at_once(gb, streams, D):
    """About 15, 36, 76 and 152 clusters of 8, 4, 2 and 1 CTAs run at once on 152 SMs."""
    lens = tuple(int(x) for x in np.random.default_rng(streams).integers(0, 120, streams))
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(streams, 3, 1, 1, lens, D, 98, page_size=16,
                                                        poison=True)
    tw, lse = t(w), torch.zeros((streams, 3, 1), device=DEV)
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), lse=lse, weights=tw)
    plain = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens))
    assert gb.device_status() == 0
    ref = OP.decode(q, kp, vp, table, lens, inputs.softmax_scale(D))
    # scores off by D products' rounding, a probability by a relative e; o by half a step of FP16
    e = 2 * (D * 2.0 ** -23 * ref["size"] + 2.0 ** -21) + 2.0 ** -20
    tol = 2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"]
    for got in (o, plain):
        assert np.all(np.abs(got.double().cpu().numpy() - ref["o"]) <= tol)
    want = w.astype(np.float64)
    for b, n in enumerate(lens):
        at = np.arange(n)
        want[table[b, at // 16], 0, at % 16] += ref["received"][b][0]
    assert np.all(np.abs(tw.double().cpu().numpy() - want) <= 2 * e.max() * 3 + 2.0 ** -23 * want)
