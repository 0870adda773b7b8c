"""Differential attention on the GPU against the float64 oracle.

Bounds.  A map's probabilities are off by the relative e of its scores (D/2 products, see
``row_error``); so the difference before the normalisation is off by at most r = c sum (p1 +
|lambda| p2) |v| with c = 2 e + 2^-22 for decode (P as two FP16 halves) and lambda's own error
(64 FP32 products and two exponentials: 2^-18 of its terms).  The normalisation divides by the
root mean square m of the row: o = x / m * g, so |o - ref| <= g (r_i / m + |x_i| rms(r) / m^2) to
first order, doubled here for the second order, plus half an FP16 step.
"""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import diff as OD

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def row_error(size):
    return 2 * ((D // 2) * 2.0 ** -23 * size + 2.0 ** -21) + 2.0 ** -20


def assert_diff(o, lse, ref, norm, lambda_init, p_step, eps=1e-5):
    """p_step: the relative step of P in the PV product, 2^-22 or 2^-11."""
    e = row_error(ref["size"])
    r = (2 * e[..., None] + p_step + 2.0 ** -18) * ref["spread"] + 2.0 ** -24
    if norm is not None:
        g = np.abs(np.asarray(norm, dtype=np.float64) * (1 - lambda_init))
        m = np.sqrt((ref["raw"] ** 2).mean(-1, keepdims=True) + eps)
        r = 2 * g * (r / m + np.abs(ref["raw"]) * np.sqrt((r * r).mean(-1, keepdims=True)) / m ** 2)
    tol = r + 2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25
    excess = np.abs(o.double().cpu().numpy() - ref["o"]) - tol
    assert np.all(excess <= 0), f"o: {int((~(excess <= 0)).sum())} outside, {np.nanmax(excess):.3e}"
    if lse is not None:
        got = lse.double().cpu().numpy()
        empty = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(got), empty)
        want = np.where(empty, 0.0, ref["lse"])
        bound = e[..., None, :] + 2.0 ** -23 * np.abs(want)
        assert np.all(np.abs(np.where(empty, 0.0, got) - want) <= bound)


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("Hq,Hkv,nq", [(1, 1, 1), (4, 1, 1), (8, 2, 1), (5, 1, 1), (6, 2, 3),
                                       (16, 1, 1), (9, 1, 2)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_decode(gb, Hq, Hkv, nq, norm):
    """Rows below, at and above one row group; lengths down to one and none (rows that see
    nothing); NaN wherever no sequence holds a row."""
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(4, Hq, Hkv, nq, (700, 1, 0, 65), D, 51,
                                                        page_size=16, spare_pages=1, poison=True)
    vecs, weight = inputs.diff_inputs(Hq, D, 52, norm=norm)
    lse = torch.zeros((4, Hq, 2, nq), device=DEV)
    o = gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), t(vecs), 0.55,
                                          norm_weight=t(weight), lse=lse)
    assert gb.device_status() == 0
    ref = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.55, 0.125, weight)
    assert_diff(o, lse, ref, weight, 0.55, 2.0 ** -22)


@pytest.mark.parametrize("heads", [1, 8])
def test_diff_decode_shared_lambda_and_long_cache(gb, heads):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(2, 8, 2, 1, (9001, 300), D, 53, page_size=64,
                                                        q_std=2.0)
    vecs, weight = inputs.diff_inputs(8, D, 54, heads=heads)
    o = gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), t(vecs), 0.2,
                                          norm_weight=t(weight), eps=1e-3)
    ref = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.2, 0.125, weight, eps=1e-3)
    assert_diff(o, None, ref, weight, 0.2, 2.0 ** -22, eps=1e-3)


def test_diff_decode_equal_halves_cancel(gb):
    """q1 = q2, k1 = k2 and lambda = 1: the two maps are one and nothing is left."""
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(1, 4, 1, 1, (400,), D, 55)
    q[..., 64:], kp[..., 64:] = q[..., :64], kp[..., :64]
    zero = torch.zeros((4, 64), device=DEV)
    o = gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), zero, 1.0)
    assert o.abs().max().item() <= 2.0 ** -18


def test_diff_decode_in_a_graph(gb):
    q, kp, vp, table, lens, _ = inputs.paged_f16_inputs(2, 8, 2, 1, (500, 90), D, 56)
    vecs, weight = inputs.diff_inputs(8, D, 57)
    args, weight = [t(x) for x in (q, kp, vp, table, lens, vecs)], t(weight)
    o = torch.empty_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gb.attn_diff_paged_decode_f16_fwd(*args, 0.3, norm_weight=weight, o=o)
    args[4].copy_(t(np.array([3, 96], dtype=np.int32)))
    graph.replay()
    want = gb.attn_diff_paged_decode_f16_fwd(*args, 0.3, norm_weight=weight)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
