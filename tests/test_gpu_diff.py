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


# ---------------------------------------------------------------- prompts

def prompt(B, Hq, Hkv, Sq, Skv, seed, std=1.0):
    q = inputs._normal_fp16(np.random.default_rng([seed, 1]), (B, Hq, Sq, D), std)
    k = inputs._normal_fp16(np.random.default_rng([seed, 2]), (B, Hkv, Skv, D))
    v = inputs._normal_fp16(np.random.default_rng([seed, 3]), (B, Hkv, Skv, D))
    return q, k, v


def check_prompt(gb, q, k, v, norm=True, lambda_init=0.55, seed=61, heads=None, workspace=None, **kw):
    B, Hq, Sq, _ = q.shape
    vecs, weight = inputs.diff_inputs(Hq, D, seed, heads=heads, norm=norm)
    lse = torch.full((B, Hq, 2, Sq), 7.0, device=DEV)
    lens = {n: None if kw.get(n) is None else t(np.asarray(kw[n], dtype=np.int32))
            for n in ("q_lens", "kv_lens")}
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), lambda_init, norm_weight=t(weight),
                                 causal=kw.get("causal", True), lse=lse, workspace=workspace, **lens)
    assert gb.device_status() == 0
    ref = OD.prefill(q, k, v, vecs, lambda_init, 0.125, weight, causal=kw.get("causal", True),
                     q_lens=kw.get("q_lens"), kv_lens=kw.get("kv_lens"))
    # P enters the PV product as one FP16 value: half a step, 2^-11 / 2, of each
    assert_diff(o, lse, ref, weight, lambda_init, 2.0 ** -11)
    return o


@pytest.mark.parametrize("Sq,Skv", [(1, 1), (1, 129), (2, 300), (64, 64), (127, 127), (128, 128),
                                    (129, 129), (130, 515), (257, 1000), (500, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_diff_prompt_lengths(gb, Sq, Skv, causal):
    """One row and one key, tile edges, a prefix, and more queries than keys (rows that see none)."""
    check_prompt(gb, *prompt(1, 2, 1, Sq, Skv, 62), causal=causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (5, 5), (8, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_prompt_heads(gb, Hq, Hkv, norm):
    check_prompt(gb, *prompt(2, Hq, Hkv, 200, 333, 63), norm=norm, heads=1 if Hq == 5 else None)


@pytest.mark.parametrize("causal", [True, False])
def test_diff_prompt_padded_batch(gb, causal):
    """Ragged lengths, empty entries, and NaN in every padded row of q, k and v."""
    q, k, v = prompt(6, 2, 1, 260, 400, 64)
    q_lens, kv_lens = [260, 100, 0, 1, 40, 200], [400, 130, 57, 0, 17, 200]
    for b in range(6):
        q[b, :, q_lens[b]:] = np.nan
        k[b, :, kv_lens[b]:] = np.nan
        v[b, :, kv_lens[b]:] = np.inf
    check_prompt(gb, q, k, v, q_lens=q_lens, kv_lens=kv_lens, causal=causal)


@pytest.mark.parametrize("Sq,Skv,q_len,kv_len", [(200, 100, 200, 100), (128, 3000, 60, 2900)])
@pytest.mark.parametrize("norm", [True, False])
def test_diff_prompt_rows_that_see_nothing_beside_an_infinite_value(gb, Sq, Skv, q_len, kv_len, norm):
    """Rows before the first key, and padding rows of a split call, share key tiles with rows that
    see an infinite value."""
    q, k, v = prompt(1, 2, 1, Sq, Skv, 71)
    v[:, :, 5] = np.inf
    vecs, weight = inputs.diff_inputs(2, D, 71, norm=norm)
    lse = torch.zeros((1, 2, 2, Sq), device=DEV)
    lens = [t(np.array([n], dtype=np.int32)) for n in (q_len, kv_len)]
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.5, norm_weight=t(weight), lse=lse,
                                 q_lens=lens[0], kv_lens=lens[1])
    assert gb.device_status() == 0
    i = np.arange(Sq)
    visible = np.where(i < q_len, np.maximum(kv_len - q_len + i + 1, 0), 0)
    none, all_of_it = t(visible == 0), t(visible > 5)
    assert none.any() and torch.all(o[:, :, none] == 0)
    assert torch.all(torch.isneginf(lse[..., none]))
    assert not torch.isfinite(o[:, :, all_of_it]).any()


def test_diff_prompt_split_keys(gb):
    """Few rows against many keys: with the full workspace, and with too little to split."""
    case = prompt(1, 2, 1, 70, 5000, 65, std=2.0)
    n = gb.attn_diff_prefill_workspace_size(1, 2, 70, 5000, D)
    assert n > 0
    for size in (n, n // 2, 16):
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        check_prompt(gb, *case, workspace=ws)
    check_prompt(gb, *prompt(3, 2, 2, 140, 3000, 66), q_lens=[140, 3, 139], kv_lens=[3000, 900, 0])


def test_diff_prompt_peaked_and_flat_scores(gb):
    for std in (0.02, 6.0):
        check_prompt(gb, *prompt(1, 2, 2, 300, 300, 67, std=std))


def test_diff_prompt_growing_scores_rescale(gb):
    """Keys whose scores climb from tile to tile: the running max moves in both maps."""
    q, k, v = prompt(1, 1, 1, 128, 1024, 68)
    q[:] = np.abs(q)
    k *= np.linspace(0.0, 3.0, 1024)[None, None, :, None].astype(np.float16)
    k[..., :64] = np.abs(k[..., :64])
    check_prompt(gb, q, k, v, causal=False)


def test_diff_prompt_strided_views(gb):
    """Token-major q and o, k and v as slices of one packed tensor."""
    q, k, v = prompt(2, 4, 2, 150, 150, 69)
    want = check_prompt(gb, q, k, v)
    tq = t(q).permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    packed = torch.zeros((2, 150, 2, 2, D), dtype=torch.float16, device=DEV)
    packed[:, :, 0], packed[:, :, 1] = t(k).permute(0, 2, 1, 3), t(v).permute(0, 2, 1, 3)
    tk, tv = (packed[:, :, i].permute(0, 2, 1, 3) for i in range(2))
    o = torch.zeros((2, 150, 4, D), dtype=torch.float16, device=DEV).permute(0, 2, 1, 3)
    vecs, weight = inputs.diff_inputs(4, D, 61)
    gb.attn_diff_prefill_fwd(tq, tk, tv, t(vecs), 0.55, norm_weight=t(weight), o=o)
    assert torch.equal(o, want)


def test_diff_prompt_many_query_tiles(gb):
    """More query tiles than SMs: several rounds of whole tiles, ragged lengths, empty entries and
    rows without keys among them."""
    q, k, v = prompt(5, 8, 4, 900, 950, 74)
    check_prompt(gb, q, k, v, q_lens=[900, 513, 0, 1, 700], kv_lens=[950, 400, 30, 0, 700])
    check_prompt(gb, q[:, :, :640], k, v, causal=False)


@pytest.mark.parametrize("split", [True, False])
def test_diff_prompt_in_a_graph_and_on_a_side_stream(gb, split):
    q, k, v = prompt(2, 2, 1, 100, 6000 if split else 200, 75)
    vecs, weight = inputs.diff_inputs(2, D, 76)
    assert (gb.attn_diff_prefill_workspace_size(2, 2, 100, k.shape[2], D) > 0) == split
    args = [t(x) for x in (q, k, v, vecs)]
    weight, lens = t(weight), t(np.array([k.shape[2], 150], dtype=np.int32))
    call = lambda **kw: gb.attn_diff_prefill_fwd(*args, 0.4, norm_weight=weight, kv_lens=lens, **kw)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    want = call()
    torch.cuda.synchronize()
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.graph(graph):
        o = call()
    lens.copy_(t(np.array([77, k.shape[2]], dtype=np.int32)))
    graph.replay()
    torch.cuda.synchronize()
    got = o.clone()
    assert torch.equal(got, call()) and not torch.equal(got, want) and gb.device_status() == 0


def test_diff_prompt_bad_length_and_lost_load(gb):
    q, k, v = prompt(2, 1, 1, 100, 100, 70)
    vecs, _ = inputs.diff_inputs(1, D, 61)
    bad = t(np.array([100, 101], dtype=np.int32))
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.5, kv_lens=bad)
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    assert torch.all(o[1] == 0) and torch.any(o[0] != 0)
    gb.set_wait_limit_ns(20_000_000)
    try:
        for mode in (1, 2):
            gb.test_inject_fault(mode)
            # no workspace to split into: mode 2 stops after 8 of the one CTA's 32 K/V tiles
            gb.attn_diff_prefill_fwd(*(t(x) for x in prompt(1, 1, 1, 128, 2048, 71)), t(vecs), 0.5,
                                     workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
            assert gb.device_status() & gb.DEV_WAIT_TIMEOUT
    finally:
        gb.test_inject_fault(0)
        gb.set_wait_limit_ns(1_000_000_000)
    check_prompt(gb, q, k, v)


def test_diff_prompt_then_decode_agree(gb):
    """The last prompt row equals one decode step over the same keys in pages."""
    B, Hq, Hkv, S, ps = 2, 4, 2, 290, 32
    q, k, v = prompt(B, Hq, Hkv, S, S, 72)
    vecs, weight = inputs.diff_inputs(Hq, D, 73)
    o = gb.attn_diff_prefill_fwd(t(q), t(k), t(v), t(vecs), 0.4, norm_weight=t(weight))
    P = B * 10
    kp, vp = torch.zeros((2, P, ps, Hkv, D), dtype=torch.float16, device=DEV)
    table = torch.randperm(P, device=DEV).to(torch.int32).reshape(B, 10).contiguous()
    lens = t(np.full(B, S, dtype=np.int32))
    gb.kv_paged_append_f16(t(k), t(v), kp, vp, table, lens)
    d = gb.attn_diff_paged_decode_f16_fwd(t(q[:, :, -1:]), kp, vp, table, lens, t(vecs), 0.4,
                                          norm_weight=t(weight))
    ref = OD.prefill(q[:, :, -1:], k, v, vecs, 0.4, 0.125, weight)
    assert_diff(o[:, :, -1:], None, ref, weight, 0.4, 2.0 ** -11)
    assert_diff(d, None, ref, weight, 0.4, 2.0 ** -22)


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


def test_wrappers_refuse_wrong_tensors(gb):
    q, k, v = (t(x) for x in prompt(2, 2, 1, 9, 17, 72))
    vecs, weight = (t(x) for x in inputs.diff_inputs(2, D, 72))
    lens = t(np.array([9, 5], dtype=np.int32))
    pages = torch.zeros((3, 16, 1, D), dtype=torch.float16, device=DEV)
    table = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    calls = [(gb.attn_diff_prefill_fwd, (q, k, v, vecs, 0.5, weight, 1e-5, True, lens, lens,
                                         torch.empty_like(q))),
             (gb.attn_diff_paged_decode_f16_fwd, (q, pages, pages, table, lens, vecs, 0.5, weight,
                                                  1e-5, None, torch.empty_like(q)))]
    for call, args in calls:
        for i, x in enumerate(args):
            if not isinstance(x, torch.Tensor):
                continue
            wider = x.double() if x.is_floating_point() else x.long()
            for wrong in (x.cpu(), wider, x[..., :-1], x[:1].clone(), x[None]):
                with pytest.raises(ValueError):
                    call(*args[:i], wrong, *args[i + 1:])
    assert gb.device_status() == 0
