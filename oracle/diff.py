"""Differential attention in float64.

Test infrastructure only (see ``oracle/__init__.py``).

A differential head splits q and k into halves and takes the difference of two
softmax maps over one set of values: o = (p1 - lambda_h p2) v, with
lambda_h = exp(lq1 . lk1) - exp(lq2 . lk2) + lambda_init from four learned
vectors, optionally normalised over the head width (root mean square, a learned
weight and the factor 1 - lambda_init).
"""

import numpy as np

from .paged import slot_rows, softmax_rows


def lambdas(vecs, lambda_init, Hq):
    """lambda of every query head: vecs [4][1 or Hq][d] in the order lq1, lk1, lq2, lk2."""
    v = np.asarray(vecs, dtype=np.float64)
    lam = np.exp((v[0] * v[1]).sum(-1)) - np.exp((v[2] * v[3]).sum(-1)) + lambda_init
    return np.broadcast_to(lam, (Hq,))


def attend(q, k, v, visible, lam, scale, norm=None, eps=1e-5, lambda_init=0.0):
    """One head: q [n][D], k, v [keys][D], visible [n][keys] bool.

    Returns (o [n][D], lse [2][n], raw [n][D], spread [n][D], size [n]): raw is o before the
    normalisation, spread = sum of (p1 + |lambda| p2) |v|, size the largest scale sum |q_i k_i|."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, D = q.shape
    d = D // 2
    raw, spread = np.zeros((n, D)), np.zeros((n, D))
    lse, size = np.full((2, n), -np.inf), np.zeros(n)
    for i in range(n):
        see = visible[i]
        if not see.any():
            continue
        for m, (part, factor) in enumerate(((slice(0, d), 1.0), (slice(d, D), -lam))):
            p, lse[m, i] = softmax_rows(k[see][:, part] @ q[i, part] * scale)
            raw[i] += factor * (p @ v[see])
            spread[i] += abs(factor) * (p @ np.abs(v[see]))
            size[i] = max(size[i], np.max(np.abs(k[see][:, part]) @ np.abs(q[i, part])) * scale)
    o = raw
    if norm is not None:
        o = raw / np.sqrt((raw * raw).mean(-1, keepdims=True) + eps)
        o = o * np.asarray(norm, dtype=np.float64) * (1.0 - lambda_init)
    return o, lse, raw, spread, size


def _all_heads(q, k, v, visible, vecs, lambda_init, scale, norm, eps):
    """q [Hq][n][D]; k, v [keys][Hkv][D]: dict of o [Hq][n][D], lse [Hq][2][n], raw, spread, size."""
    Hq = q.shape[0]
    grp = Hq // k.shape[1]
    lam = lambdas(vecs, lambda_init, Hq)
    heads = [attend(q[h], k[:, h // grp], v[:, h // grp], visible, lam[h], scale, norm, eps,
                    lambda_init) for h in range(Hq)]
    return {name: np.stack([x[j] for x in heads])
            for j, name in enumerate(("o", "lse", "raw", "spread", "size"))}


def _stack(parts):
    return {name: np.stack([p[name] for p in parts]) for name in parts[0]}


def prefill(q, k, v, vecs, lambda_init, scale, norm=None, eps=1e-5, causal=True, q_lens=None,
            kv_lens=None):
    """q [B][Hq][Sq][D]; k, v [B][Hkv][Skv][D].  Query i < q_lens[b] sits at position
    kv_lens[b] - q_lens[b] + i and sees the keys up to it (causal) or all kv_lens[b]; later
    query rows see nothing."""
    B, Hq, Sq, D = q.shape
    Skv = k.shape[2]
    parts = []
    for b in range(B):
        ql = Sq if q_lens is None else int(q_lens[b])
        kl = Skv if kv_lens is None else int(kv_lens[b])
        i, t = np.arange(Sq)[:, None], np.arange(Skv)[None, :]
        visible = (t < kl) & (i < ql)
        if causal:
            visible &= t <= kl - ql + i
        parts.append(_all_heads(q[b], k[b].transpose(1, 0, 2), v[b].transpose(1, 0, 2), visible,
                                vecs, lambda_init, scale, norm, eps))
    return _stack(parts)


def paged_decode(q, k_pages, v_pages, table, kv_lens, vecs, lambda_init, scale, norm=None,
                 eps=1e-5):
    """q [B][Hq][nq][D] over FP16 pages; query i sees the tokens t <= kv_lens[b] - nq + i."""
    nq = q.shape[2]
    parts = []
    for b in range(q.shape[0]):
        n = int(kv_lens[b])
        k, v = slot_rows(k_pages, table[b], n), slot_rows(v_pages, table[b], n)
        visible = np.arange(n)[None, :] <= (n - nq + np.arange(nq))[:, None]
        parts.append(_all_heads(q[b], k, v, visible, vecs, lambda_init, scale, norm, eps))
    return _stack(parts)
