"""Differential prompts whose two maps resemble each other, against the float64 oracle: what they have
in common cancels, and the rounding of the probabilities must not be what is left.

Bounds.  As for the other differential prompts, with the probabilities as FP16 hi + lo halves: a
relative 2^-22 (half a step of FP16 is 2^-11, twice).  Small queries make the scores' own error, e,
as small as that: probabilities held in one FP16 value are off by up to 2^-11, far outside.
"""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import diff as OD

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def row_error(size, terms):
    return 2 * (terms * 2.0 ** -23 * size + 2.0 ** -21) + 2.0 ** -20


def within(got, ref, tol):
    excess = np.abs(got.double().cpu().numpy() - ref) - tol
    assert np.all(excess <= 0), f"{int((~(excess <= 0)).sum())} outside, worst {np.nanmax(excess):.3e}"


def check_diff(o, lse, ref, norm, lambda_init, eps=1e-5):
    """As the differential tests': r bounds the difference before the norm, the norm divides it by
    the row's root mean square."""
    e = row_error(ref["size"], 64)
    r = (2 * e[..., None] + 2.0 ** -22 + 2.0 ** -18) * ref["spread"] + 2.0 ** -24
    if norm is not None:
        g = np.abs(np.asarray(norm, dtype=np.float64) * (1 - lambda_init))
        m = np.sqrt((ref["raw"] ** 2).mean(-1, keepdims=True) + eps)
        r = 2 * g * (r / m + np.abs(ref["raw"]) * np.sqrt((r * r).mean(-1, keepdims=True)) / m ** 2)
    within(o, ref["o"], r + 2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25)
    within(lse, ref["lse"], e[..., None, :] + 2.0 ** -23 * np.abs(ref["lse"]))


def alike(shape, std, alpha, seed):
    """Rows [.., 128] whose second half is the first but for a part sqrt(1 - alpha^2)."""
    rng = np.random.default_rng(seed)
    a, b = rng.standard_normal((2,) + shape[:-1] + (64,))
    return (std * np.concatenate([a, alpha * a + np.sqrt(1 - alpha ** 2) * b], -1)).astype(np.float16)


@pytest.mark.parametrize("Sq,Skv,std", [(1, 24, 0.05), (60, 60, 0.05), (40, 2000, 1.0)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_prompt_of_maps_that_resemble_each_other(gb, Sq, Skv, std, norm):
    """What the maps have in common cancels: P is rounded far below the output's own step."""
    q, k = alike((1, 2, Sq, 128), std, 0.999, 87), alike((1, 1, Skv, 128), 1.0, 0.999, 88)
    v = inputs._normal_fp16(np.random.default_rng(89), (1, 1, Skv, 128))
    vecs, weight = inputs.diff_inputs(2, 128, 90, norm=norm)
    lse = torch.zeros((1, 2, 2, Sq), device=DEV)
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.9, norm_weight=t(weight), causal=False,
                                 lse=lse)
    assert gb.device_status() == 0
    check_diff(o, lse, OD.prefill(q, k, v, vecs, 0.9, 0.125, weight, causal=False), weight, 0.9)
