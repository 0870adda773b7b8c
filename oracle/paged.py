"""The FP16 page cache in float64: append, decode with accumulated weights, eviction.

Test infrastructure only (see ``oracle/__init__.py``).

The page format is the E4M3 cache's ("Integrate FP32 v37 prefill and exact E4M3
bridge", Implementation: pages and page table) with FP16 elements: a pool
[num_phys_pages][page_size][Hkv][D] and one page-table row per sequence.  The
attention weight of a cached token and KV head is the sum of the softmax
probabilities it received from every query head of the group, added up over
the calls; eviction keeps, per KV head, the first tokens, the newest and the
heaviest of the rest.
"""

import numpy as np


def slot_rows(pages, table_row, n):
    """The first n cached rows of a sequence: [n][Hkv][D]."""
    ps = pages.shape[1]
    t = np.arange(n)
    return pages[np.asarray(table_row)[t // ps], t % ps]


def append(k_new, v_new, k_pages, v_pages, table, kv_lens, new_lens=None, weights=None):
    """Copies of (k_pages, v_pages, weights) with the new tokens written: k_new, v_new
    [B][Hkv][n][D]; token i of sequence b goes to slot kv_lens[b] - new_lens[b] + i."""
    k_pages, v_pages = k_pages.copy(), v_pages.copy()
    weights = None if weights is None else weights.copy()
    ps = k_pages.shape[1]
    B, _, n, _ = k_new.shape
    for b in range(B):
        count = n if new_lens is None else int(new_lens[b])
        for i in range(count):
            t = int(kv_lens[b]) - count + i
            page, slot = table[b, t // ps], t % ps
            k_pages[page, slot] = k_new[b, :, i]
            v_pages[page, slot] = v_new[b, :, i]
            if weights is not None:
                weights[page, :, slot] = 0
    return k_pages, v_pages, weights


def softmax_rows(x):
    """(probabilities, log of the sum of exponentials) of one row; all -inf: zeros and -inf."""
    m = np.max(x) if x.size else -np.inf
    if m == -np.inf:
        return np.zeros_like(x), -np.inf
    e = np.exp(x - m)
    return e / e.sum(), m + np.log(e.sum())


def decode(q, k_pages, v_pages, table, kv_lens, scale):
    """Decode attention over FP16 pages.

    q [B][Hq][nq][D]; query i of sequence b sees the tokens t <= kv_lens[b] - nq + i.
    Returns a dict of float64 arrays: o [B][Hq][nq][D], lse [B][Hq][nq], received (list over b of
    [Hkv][kv_lens[b]]: the probabilities each token received), spread (sum of p |v|, like o) and
    size (largest sum_i |q_i k_i| scale of a row, like lse), from which error bounds follow."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, nq, D = q.shape
    Hkv = k_pages.shape[2]
    grp = Hq // Hkv
    out = {"o": np.zeros((B, Hq, nq, D)), "lse": np.full((B, Hq, nq), -np.inf),
           "spread": np.zeros((B, Hq, nq, D)), "size": np.zeros((B, Hq, nq)), "received": []}
    for b in range(B):
        n = int(kv_lens[b])
        k = slot_rows(k_pages, table[b], n).astype(np.float64)
        v = slot_rows(v_pages, table[b], n).astype(np.float64)
        got = np.zeros((Hkv, n))
        for h in range(Hq):
            for i in range(nq):
                m = n - nq + i + 1
                if m <= 0:
                    continue
                kh, vh = k[:m, h // grp], v[:m, h // grp]
                p, out["lse"][b, h, i] = softmax_rows(kh @ q[b, h, i] * scale)
                out["o"][b, h, i] = p @ vh
                out["spread"][b, h, i] = p @ np.abs(vh)
                out["size"][b, h, i] = np.max(np.abs(kh) @ np.abs(q[b, h, i])) * scale
                got[h // grp, :m] += p
        out["received"].append(got)
    return out


def evict_kept(weights, n, budget, sink, recent):
    """Slots kept of n cached tokens of one KV head with the given weights [n], ascending."""
    if n <= budget:
        return np.arange(n)
    w = np.where(np.isnan(weights), -np.inf, np.asarray(weights, dtype=np.float64))
    nan = np.isnan(weights)
    middle = range(sink, n - recent)
    order = sorted(middle, key=lambda t: (-w[t], nan[t], t))   # a NaN after -inf; ties: lower slot
    keep = list(range(sink)) + sorted(order[:budget - sink - recent]) + \
        list(range(n - recent, n))
    return np.array(keep, dtype=np.int64)


def evict(k_pages, v_pages, weights, table, dst_table, kv_lens, budget, sink, recent):
    """(k_pages, v_pages, weights, new_lens, kept) after the eviction; rows kept by KV head h move
    to slots 0.. of dst_table's pages."""
    src_k, src_v, src_w = k_pages, v_pages, weights
    k_pages, v_pages, weights = k_pages.copy(), v_pages.copy(), weights.copy()
    ps, Hkv = k_pages.shape[1], k_pages.shape[2]
    B = len(kv_lens)
    kept = np.full((B, Hkv, budget), -1, dtype=np.int32)
    for b in range(B):
        n = int(kv_lens[b])
        t = np.arange(n)
        page, slot = table[b, t // ps], t % ps
        for h in range(Hkv):
            keep = evict_kept(src_w[page, h, slot], n, budget, sink, recent)
            kept[b, h, :len(keep)] = keep
            j = np.arange(len(keep))
            to, at = dst_table[b, j // ps], j % ps
            k_pages[to, at, h] = src_k[page[keep], slot[keep], h]
            v_pages[to, at, h] = src_v[page[keep], slot[keep], h]
            weights[to, h, at] = src_w[page[keep], h, slot[keep]]
    return k_pages, v_pages, weights, np.minimum(kv_lens, budget).astype(np.int32), kept
