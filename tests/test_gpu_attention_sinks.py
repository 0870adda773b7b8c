"""What becomes of probabilities far below the largest, beside attention sinks, against the float64
oracle.

Bounds.  The PV product takes a probability as two FP16 halves of p' = 2^(x - reference + SHIFT), a
relative 2^-22 while p' is well inside FP16's range and an absolute 2^-25 below.  The reference is at
most the row's largest score, so the row's sum of p' is at least 2^SHIFT sum 2^(x - max) and the
small ones move an output by at most 2^-(25 + SHIFT) sum |v| / sum 2^(x - max).  The other terms
are those of the decode and prompt tests: a probability is off by a relative e from its score
(D products), O by half a step of FP16.
"""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import diff as OD
from oracle import paged as OP

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHIFT = 11
TAIL = 25.5 * np.log(2.0)   # a sink's score above the others': they are below FP16's last half step


def t(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def row_error(size, terms):
    return 2 * (terms * 2.0 ** -23 * size + 2.0 ** -21) + 2.0 ** -20


def within(got, ref, tol):
    excess = np.abs(got.double().cpu().numpy() - ref) - tol
    assert np.all(excess <= 0), f"{int((~(excess <= 0)).sum())} outside, worst {np.nanmax(excess):.3e}"


def sink_rows(n, every, heads, D, maps, seed):
    """Keys whose every `every`-th has the score TAIL (in each map, for q = 1) and value 0, the others
    score 0 and values of one sign."""
    k = np.zeros((n, heads, D), dtype=np.float16)
    k[::every] = TAIL / np.sqrt(D // maps)
    v = np.random.default_rng(seed).uniform(800, 1600, (n, heads, D)).astype(np.float16)
    v[::every] = 0
    return k, v


def small_step(v, every):
    """The bound on what the smallest probabilities lose: v [n][heads][D] of one sequence."""
    n = v.shape[0]
    sinks = -(-n // every)
    return 2.0 ** -(25 + SHIFT) * np.abs(v.astype(np.float64)).sum(0) / sinks


def sink_pages(lens, Hq, Hkv, nq, D, maps, seed, max_kv):
    ps = 16
    q, kp, vp, table, lens, w = inputs.paged_f16_inputs(len(lens), Hq, Hkv, nq, lens, D, seed,
                                                        page_size=ps)
    q[:] = 1
    for b, n in enumerate(lens):
        k, v = sink_rows(n, 16, Hkv, D, maps, seed + b)
        at = np.arange(n)
        kp[table[b, at // ps], at % ps], vp[table[b, at // ps], at % ps] = k, v
    if max_kv is not None:
        wide = np.full((len(lens), max_kv // ps), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    small = np.stack([small_step(OP.slot_rows(vp, table[b], n), 16) for b, n in enumerate(lens)])
    return q, kp, vp, table, lens, w, np.repeat(small, Hq // Hkv, 1)[:, :, None]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_kv", [None, 300000])   # in clusters where D allows, and end to end
def test_decode_beside_attention_sinks(gb, D, max_kv):
    q, kp, vp, table, lens, w, small = sink_pages((1500, 700, 16), 4, 2, 1, D, 1, 81, max_kv)
    lse, tw = torch.zeros((3, 4, 1), device=DEV), t(np.zeros_like(w))
    o = gb.attn_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), lse=lse, weights=tw)
    assert gb.device_status() == 0
    ref = OP.decode(q, kp, vp, table, lens, inputs.softmax_scale(D))
    e = row_error(ref["size"], D)
    within(o, ref["o"], 2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + small +
           (2 * e[..., None] + 2.0 ** -21) * ref["spread"])
    within(lse, ref["lse"], e + 2.0 ** -23 * np.abs(ref["lse"]))
    want, tol = np.zeros(w.shape), np.zeros(w.shape)
    for b, n in enumerate(lens):
        at = np.arange(n)
        for h in range(2):
            want[table[b, at // 16], h, at % 16] = ref["received"][b][h]
    within(tw, want, (2 * e.max() + 2.0 ** -22) * want + 2.0 ** -100)


@pytest.mark.parametrize("max_kv", [None, 300000])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_decode_beside_attention_sinks(gb, max_kv, norm):
    q, kp, vp, table, lens, _, small = sink_pages((1500, 700, 16), 4, 2, 2, 128, 2, 83, max_kv)
    vecs, weight = inputs.diff_inputs(4, 128, 84, norm=norm)
    lse = torch.zeros((3, 4, 2, 2), device=DEV)
    o = gb.attn_diff_paged_decode_f16_fwd(t(q), t(kp), t(vp), t(table), t(lens), t(vecs), 0.3,
                                          norm_weight=t(weight), eps=1e-9, lse=lse)
    assert gb.device_status() == 0
    ref = OD.paged_decode(q, kp, vp, table, lens, vecs, 0.3, 0.125, weight, eps=1e-9)
    check_diff(o, lse, ref, weight, 0.3, 2 * small, eps=1e-9)


def check_diff(o, lse, ref, norm, lambda_init, small=0.0, eps=1e-5):
    """As the differential tests': r bounds the difference before the norm, the norm divides it by
    the row's root mean square."""
    e = row_error(ref["size"], 64)
    r = (2 * e[..., None] + 2.0 ** -22 + 2.0 ** -18) * ref["spread"] + small + 2.0 ** -24
    if norm is not None:
        g = np.abs(np.asarray(norm, dtype=np.float64) * (1 - lambda_init))
        m = np.sqrt((ref["raw"] ** 2).mean(-1, keepdims=True) + eps)
        r = 2 * g * (r / m + np.abs(ref["raw"]) * np.sqrt((r * r).mean(-1, keepdims=True)) / m ** 2)
    within(o, ref["o"], r + 2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25)
    within(lse, ref["lse"], e[..., None, :] + 2.0 ** -23 * np.abs(ref["lse"]))


@pytest.mark.parametrize("Sq,Skv", [(200, 200), (130, 5000)])   # whole query tiles, and keys split
@pytest.mark.parametrize("norm", [True, False])
def test_diff_prompt_beside_attention_sinks(gb, Sq, Skv, norm):
    k, v = (x.transpose(1, 0, 2)[None] for x in sink_rows(Skv, 64, 2, 128, 2, 85))
    q = np.ones((1, 4, Sq, 128), dtype=np.float16)
    vecs, weight = inputs.diff_inputs(4, 128, 86, norm=norm)
    lse = torch.zeros((1, 4, 2, Sq), device=DEV)
    assert (gb.attn_diff_prefill_workspace_size(1, 4, Sq, Skv, 128) > 0) == (Skv == 5000)
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.3, norm_weight=t(weight), eps=1e-9,
                                 causal=False, lse=lse)
    assert gb.device_status() == 0
    ref = OD.prefill(q, k, v, vecs, 0.3, 0.125, weight, eps=1e-9, causal=False)
    small = np.repeat(small_step(v[0].transpose(1, 0, 2), 64), 2, 0)[None, :, None]
    check_diff(o, lse, ref, weight, 0.3, 2 * small, eps=1e-9)
