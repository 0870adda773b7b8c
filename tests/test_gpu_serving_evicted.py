"""Requests that go on after an eviction: the tokens that stay keep the rotation of the places where they came, so
the next tokens' positions are their places in the text -- kv_paged_extend's, which count what the cache
holds, and what the sequence has lost."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP, rope as OR
from tests.test_gpu_paged_f16 import assert_within, row_error
from tests.test_gpu_rope import close

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("captured", [False, True])
def test_positions_after_evictions(gb, captured):
    rng = np.random.default_rng(11)
    B, Hq, Hkv, D, ps, P, budget, steps = 2, 4, 2, 64, 16, 40, 48, 5
    scale = inputs.softmax_scale(D)
    freqs = gb.rope_frequencies(D)
    f = freqs.cpu().numpy()
    kp, vp = (torch.zeros((P, ps, Hkv, D), dtype=torch.float16, device=DEV) for _ in range(2))
    weights = torch.zeros((P, Hkv, ps), device=DEV)
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    free, count = i32(rng.permutation(P)), i32([P])
    lens, lost = i32([0, 0]), i32([0, 0])
    texts = [[], []]                                  # every token's key and value [Hkv][2][D]
    held = [[[] for _ in range(Hkv)] for _ in range(B)]   # places in the text of what each KV head's cache holds

    def come(new, n):
        """Host tokens, padded to n a row: q, k, v [B][H][n][D]."""
        q, k, v = (rng.standard_normal((B, h, n, D)).astype(np.float16) for h in (Hq, Hkv, Hkv))
        for b, m in enumerate(new):
            at = len(texts[b])
            texts[b] += [(k[b, :, i], v[b, :, i]) for i in range(m)]
            held[b] = [h + list(range(at, at + m)) for h in held[b]]
        return q, k, v

    def step(q, k, v, new):
        _, _, _, places, slots = gb.kv_paged_extend(table, lens, new, free, count, ps, P, row_tokens=q.shape[2],
                                                    kv_lens_out=lens, free_count_out=count)
        positions = torch.where(places >= 0, places + lost[:, None], places)
        turned = gb.kv_paged_rope_append(q, k, v, slots, kp, vp, positions, freqs, weights=weights)
        return turned, gb.attn_paged_decode_f16_fwd(turned, kp, vp, table, lens, weights=weights)

    def check_cache():
        tab, k, v = table.cpu().numpy(), kp.cpu().numpy(), vp.cpu().numpy()
        for b in range(B):
            for h in range(Hkv):
                where = np.array(held[b][h])
                s = np.arange(len(where))
                at = tab[b, s // ps], s % ps, h
                want = np.stack([texts[b][w][0][h] for w in where])[None, None]
                ref, size = OR.rotate(want, where[None, None], f)
                close(k[at], ref[0, 0], size[0, 0], f"keys {b}, {h}")
                assert np.array_equal(v[at], np.stack([texts[b][w][1][h] for w in where]))

    new = [130, 40]
    q, k, v = come(new, 130)
    step(*(torch.from_numpy(x).to(DEV) for x in (q, k, v)), i32(new))
    assert lens.tolist() == new
    one = i32([1, 1])
    bufs = [torch.zeros((B, h, 1, D), dtype=torch.float16, device=DEV) for h in (Hq, Hkv, Hkv)]
    graph = None
    if captured:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            outs = step(*bufs, one)
    for i in range(3 * steps):
        if i % steps == 0:                            # down to the budget, pages back
            before = lens.clone()
            new_lens, kept = gb.kv_paged_evict(kp, vp, weights, table, lens, budget, sink=4, recent=8)
            gb.kv_paged_release(table, lens, free, count, ps, P, keep_lens=new_lens, free_count_out=count)
            lost += before - new_lens
            lens.copy_(new_lens)
            kept = kept.cpu().numpy()
            for b, n in enumerate(new_lens.tolist()):
                held[b] = [[held[b][h][x] for x in kept[b, h, :n]] for h in range(Hkv)]
            check_cache()
        x = come([1, 1], 1)
        for buf, y in zip(bufs, x):
            buf.copy_(torch.from_numpy(y))
        if graph:
            graph.replay()
            turned, o = outs
        else:
            turned, o = step(*bufs, one)
        torch.cuda.synchronize()
        text = np.array([len(s) - 1 for s in texts])   # the new token's place
        ref, size = OR.rotate(x[0], text[None, :, None], f)
        close(turned.cpu().numpy(), ref, size, "queries")
        check_cache()
        qt = turned.cpu().numpy()
        ref = OP.decode(qt, kp.cpu().numpy(), vp.cpu().numpy(), table.cpu().numpy(), lens.tolist(), scale)
        e = row_error(ref["size"], D)
        assert_within(o.float().cpu().numpy(), ref["o"],
                      2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], "o")
    assert lost.tolist() == [len(s) - n for s, n in zip(texts, lens.tolist())] and lost[0] > 82
    assert gb.device_status() == 0
