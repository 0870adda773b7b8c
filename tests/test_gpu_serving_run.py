"""Serving steps from request lengths to outputs: pages and slots (kv_paged_extend), norms, rotation and
append in one call (kv_paged_rope_append), decode behind a shared prefix, pages given back
(kv_paged_release), with eviction and the E4M3 cache, against float64 oracles that are given the bytes
that the calls left in the cache."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import attention as OA, decode as OD, paged as OP, rope as OR, tables as OT
from tests.test_gpu_paged_f16 import assert_within, row_error
from tests.test_gpu_rope import close

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def attention_close(o, q, kp, vp, table, lens):
    ref = OP.decode(q, kp, vp, table, lens, inputs.softmax_scale(q.shape[3]))
    e = row_error(ref["size"], q.shape[3])
    assert_within(o.float().cpu().numpy(), ref["o"],
                  2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], "o")


def test_requests_behind_a_system_prompt(gb):
    """A prompt of 200 tokens is read in once; three requests fork from its whole pages and bring
    their own; four decoding steps; one ends, another takes its pages; all pages come back."""
    rng = np.random.default_rng(1)
    Hq, Hkv, D, ps, P, width, B = 8, 2, 128, 16, 64, 24, 4
    freqs = gb.rope_frequencies(D, factor=4.0, trained_len=128, method="turns", high_turns=4.0)
    wq, wk = (t((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
    kp = torch.zeros((P, ps, Hkv, D), dtype=torch.float16, device=DEV)
    vp = torch.zeros_like(kp)
    weights = torch.full((P, Hkv, ps), 5.0, device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    free, count = i32(rng.permutation(P)), i32([P])
    lens = i32([0, 0, 0, 0])
    host_table, host_lens, stack = table.cpu().numpy(), [0] * B, free.tolist()

    def tokens(new):
        """The new tokens' q, k, v through the calls; returns q as [1, Hq, T, D]."""
        nonlocal host_table, host_lens, stack, lens, count
        T = sum(new) + 3                                # a padded buffer, as captured steps have
        qkv = (1.5 * rng.standard_normal((1, T, Hq + 2 * Hkv, D))).astype(np.float16)
        q, k, v = (x.permute(0, 2, 1, 3) for x in t(qkv).split([Hq, Hkv, Hkv], 2))
        lens, count, starts, pos, slots = gb.kv_paged_extend(table, lens, i32(new), free, count, ps, P,
                                                             max_tokens=T)
        host_table, host_lens, stack, toks, refused = OT.extend(host_table, host_lens, new, stack, ps)
        rp, rs, _ = OT.packed(toks, T)
        assert not refused and pos.tolist() == rp.tolist() and slots.tolist() == rs.tolist()
        q = gb.kv_paged_rope_append(q, k, v, slots[None], kp, vp, pos[None], freqs, q_weight=wq,
                                    k_weight=wk, weights=weights)
        live, f = rp >= 0, freqs.cpu().numpy()
        where = np.maximum(rp, 0)[None, None]
        x = qkv.transpose(0, 2, 1, 3)
        for got, part, w in ((q, x[:, :Hq], wq), (None, x[:, Hq:Hq + Hkv], wk)):
            ref, size = OR.rotate(part, where, f, w.cpu().numpy())
            if got is None:                             # keys: from their slots
                rows = kp.reshape(-1, Hkv, D)[torch.from_numpy(rs[live].astype(np.int64)).to(DEV)]
                got = rows.cpu().numpy().transpose(1, 0, 2)[None]
            else:
                got = got.cpu().numpy()[:, :, live]
            close(got, ref[:, :, live], size[:, :, live], "rotated")
        return q[:, :, live]

    q = tokens([200, 0, 0, 0])
    attention_close(gb.attn_paged_decode_f16_fwd(q.contiguous(), kp, vp, table[:1], lens[:1]),
                    q.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(), host_table[:1], host_lens[:1])
    prefix = 192                                        # whole pages; the requests bring the rest
    for b in range(1, B):
        table[b, :prefix // ps] = table[0, :prefix // ps]
        host_table[b, :prefix // ps] = host_table[0, :prefix // ps]
        lens[b], host_lens[b] = prefix, prefix
    tokens([0, 40, 3, 17])
    starts, pre = i32([0, B]), i32([prefix])
    for step in range(4):
        q = tokens([1] * B).permute(2, 1, 0, 3).contiguous()        # [B, Hq, 1, D]
        args = (q, kp, vp, table, lens)
        o = gb.attn_paged_decode_shared_f16_fwd(*args, starts, pre)
        attention_close(o, q.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(), host_table, host_lens)
        plain = gb.attn_paged_decode_f16_fwd(*args, weights=weights)
        assert (o.float() - plain.float()).abs().max() <= 2.0 ** -10 * plain.float().abs().max()
    assert gb.device_status() == 0
    # request 2 ends: its own pages come back, the prefix stays for the others
    keep = [n if b != 2 else prefix for b, n in enumerate(host_lens)]
    count = gb.kv_paged_release(table, lens, free, count, ps, P, keep_lens=i32(keep))
    stack = OT.release(host_table, host_lens, keep, stack, ps, P)
    assert free.tolist()[:count.item()] == stack
    lens, host_lens = i32(keep), keep
    # another request in its place, behind the same prefix
    tokens([0, 0, 70, 0])
    q = tokens([1] * B).permute(2, 1, 0, 3).contiguous()
    o = gb.attn_paged_decode_shared_f16_fwd(q, kp, vp, table, lens, starts, pre)
    attention_close(o, q.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(), host_table, host_lens)
    # the requests end, then the prompt with its prefix
    for keep in ([host_lens[0]] + [prefix] * 3, [0] + [prefix] * 3):
        count = gb.kv_paged_release(table, lens, free, count, ps, P, keep_lens=i32(keep))
        stack = OT.release(host_table, host_lens, keep, stack, ps, P)
        lens, host_lens = i32(keep), keep
    assert sorted(stack) == list(range(P)) and free.tolist() == stack and count.item() == P
    assert gb.device_status() == 0


def test_captured_step_of_three_calls(gb):
    """extend, rotate and append, decode in one graph whose lengths and count live on the device."""
    rng = np.random.default_rng(2)
    B, Hq, Hkv, D, ps, P = 5, 4, 1, 64, 16, 40
    kp = torch.zeros((P, ps, Hkv, D), dtype=torch.float16, device=DEV)
    vp = torch.zeros_like(kp)
    table, free = torch.full((B, 8), -1, dtype=torch.int32, device=DEV), i32(rng.permutation(P))
    lens, count, new = i32([0] * B), i32([P]), i32([0] * B)
    freqs = gb.rope_frequencies(32)
    host_table, host_lens, stack = table.cpu().numpy(), [0] * B, free.tolist()
    n = 3
    q, k, v = (torch.empty((B, h, n, D), dtype=torch.float16, device=DEV) for h in (Hq, Hkv, Hkv))
    starts, pre = i32([0, 2, B]), i32([0, 0])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        _, _, _, pos, slots = gb.kv_paged_extend(table, lens, new, free, count, ps, P, row_tokens=n,
                                                 kv_lens_out=lens, free_count_out=count)
        turned = gb.kv_paged_rope_append(q, k, v, slots, kp, vp, pos, freqs, interleaved=True)
        o = gb.attn_paged_decode_shared_f16_fwd(turned, kp, vp, table, lens, starts, pre)
    for step in range(6):
        m = [int(x) for x in rng.integers(1, n + 1, B)] if step % 2 else [n] * B
        new.copy_(i32(m))
        for x in (q, k, v):
            x.copy_(t(rng.standard_normal(x.shape).astype(np.float16)))
        graph.replay()
        torch.cuda.synchronize()
        host_table, host_lens, stack, toks, refused = OT.extend(host_table, host_lens, m, stack, ps)
        assert not refused and lens.tolist() == host_lens and count.item() == len(stack)
        assert np.array_equal(table.cpu().numpy(), host_table)
        full = [b for b in range(B) if m[b] == n]       # the others' last rows are padding
        attention_close(o[full], turned[full].cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(),
                        host_table[full], [host_lens[b] for b in full])
    assert gb.device_status() == 0


def test_e4m3_cache_from_rotated_tokens(gb):
    """The E4M3 decode over codes that kv_paged_rope_append wrote."""
    rng = np.random.default_rng(3)
    Hq, Hkv, D, ps, P, T = 6, 1, 256, 32, 8, 170
    ks, vs = 0.03125, 0.02
    kp = torch.zeros((P, ps, Hkv, D), dtype=torch.uint8, device=DEV)
    vp = torch.zeros_like(kp)
    table = torch.full((1, P), -1, dtype=torch.int32, device=DEV)
    lens, _, _, pos, slots = gb.kv_paged_extend(table, i32([0]), i32([T]), i32(range(P)), i32([P]), ps, P,
                                                max_tokens=T)
    q, k, v = (t(rng.standard_normal((1, h, T, D)).astype(np.float16)) for h in (Hq, Hkv, Hkv))
    freqs = gb.rope_frequencies(64)
    q = gb.kv_paged_rope_append(q, k, v, slots[None], kp, vp, pos[None], freqs, k_scale=ks, v_scale=vs)
    newest = q[:, :, -2:].contiguous()
    o = gb.attn_paged_decode_fwd(newest, kp, vp, table, lens, ks, vs)
    ref, _ = OD.paged_decode_attention(newest.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy(),
                                       table.cpu().numpy(), np.array([T], dtype=np.int32), ks, vs,
                                       inputs.softmax_scale(D))
    assert_within(o.float().cpu().numpy(), ref, 2e-3 + 1e-2 * np.abs(ref), "o")
    # what the codes stand for is the rotated key within half a step
    want, size = OR.rotate(k.cpu().numpy(), pos.cpu().numpy()[None, None], freqs.cpu().numpy())
    kf, _ = gb.e4m3_paged_to_fp16(kp, vp, table[0], T, ks, vs)
    close(kf[None].cpu().numpy(), want, size, "bridged keys", 2.0 ** -4 + 2.0 ** -10, 2.0 ** -10 * ks + 2.0 ** -25)
    assert gb.device_status() == 0


def test_rotated_prompt_into_the_causal_prefill(gb):
    """Norm and rotation in place in a packed projection, then the prefill on its strided views."""
    rng = np.random.default_rng(4)
    Hq, Hkv, S, D = 6, 1, 256, 256
    qkv = rng.standard_normal((1, S, Hq + 2 * Hkv, D)).astype(np.float16)
    whole = t(qkv)
    q, k, v = (x.permute(0, 2, 1, 3) for x in whole.split([Hq, Hkv, Hkv], 2))
    w = (1 + 0.1 * rng.standard_normal(D)).astype(np.float32)
    freqs = gb.rope_frequencies(64)
    pos = torch.arange(S, dtype=torch.int32, device=DEV)[None]
    gb.qk_norm_rope_f16(q, k, pos, freqs, q_weight=t(w), k_weight=t(w), q_out=q, k_out=k)
    x = qkv.transpose(0, 2, 1, 3)
    p, f = np.arange(S)[None, None], freqs.cpu().numpy()
    for got, part in ((q, x[:, :Hq]), (k, x[:, Hq:Hq + Hkv])):
        close(got.cpu().numpy(), *OR.rotate(part, p, f, w), "rotated")
    assert np.array_equal(v.cpu().numpy(), x[:, Hq + Hkv:])
    o = gb.attn_causal_prefill_fwd(q, k, v, prob_split=True)
    ref, _ = OA.causal_prefill_attention(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(),
                                         inputs.softmax_scale(D), S)
    assert_within(o.float().cpu().numpy(), ref, 2e-3 + 1e-2 * np.abs(ref), "o")
    assert gb.device_status() == 0


def test_eviction_and_its_pages_back(gb):
    """A cache evicted in place gives back the pages behind its budget, which the next tokens take."""
    rng = np.random.default_rng(5)
    B, Hkv, D, ps, P, budget = 2, 2, 64, 16, 40, 48
    kp, vp = (t(rng.standard_normal((P, ps, Hkv, D)).astype(np.float16)) for _ in range(2))
    weights = t(rng.random((P, Hkv, ps)).astype(np.float32))
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    free, count = i32(rng.permutation(P)), i32([P])
    lens, count, _, _, _ = gb.kv_paged_extend(table, i32([0, 0]), i32([130, 40]), free, count, ps, P)
    new_lens, _ = gb.kv_paged_evict(kp, vp, weights, table, lens, budget, sink=4, recent=8)
    before = count.item()
    count = gb.kv_paged_release(table, lens, free, count, ps, P, keep_lens=new_lens)
    assert new_lens.tolist() == [48, 40] and count.item() == before + 6     # 9 pages to 3, 3 stay
    lens, count, _, pos, slots = gb.kv_paged_extend(table, new_lens, i32([20, 20]), free, count, ps, P,
                                                    row_tokens=20)
    assert lens.tolist() == [68, 60] and pos[0].tolist() == list(range(48, 68))
    pages = set(table[0, :5].tolist()) | set(table[1, :4].tolist())
    assert len(pages) == 9 and len(set(slots.flatten().tolist())) == 40 and count.item() == before + 3
    assert gb.device_status() == 0
