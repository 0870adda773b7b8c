"""The FP16 page cache (append, decode with accumulated attention weights, eviction) and
differential attention (prompts and decode): what is measured of them, and their plain forms.

`run` computes one pass of an operator from `prepare`'s state: with elementary torch operations
in FP32, or, where `own` is true, by the library's calls.  `exact` is the definition in float64.

A cache is a pool of pages k_pages, v_pages [P][page][Hkv][D] FP16 with one page-table row per
sequence; `weights` FP32 [P][Hkv][page] holds the attention weight every cached token has received
so far.
"""

import math

import torch

own = False

EPS = 1e-5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a busy server: one token for each of 64 sequences
        {"name": "append one token", "op": "append", "B": 64, "n": 1, "Hkv": 8, "D": 128,
         "page": 16, "lo": 300, "hi": 6000, "ragged": False, "weights": True},
        # prompts of four requests enter the cache
        {"name": "append prompts", "op": "append", "B": 4, "n": 8192, "Hkv": 8, "D": 128,
         "page": 64, "lo": 8192, "hi": 9001, "ragged": True, "weights": True},
        # one short conversation: latency
        {"name": "decode one short sequence", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "nq": 1, "page": 16, "lo": 511, "hi": 511, "weights": False},
        # an ordinary batch of conversations whose caches are kept within a budget
        {"name": "decode batch with weights", "op": "decode", "B": 32, "Hq": 32, "Hkv": 8,
         "D": 128, "nq": 1, "page": 16, "lo": 257, "hi": 8191, "weights": True},
        # long documents, the head layout and lengths of the benchmark's E4M3 decode
        {"name": "decode long caches", "op": "decode", "B": 4, "Hq": 6, "Hkv": 1, "D": 256,
         "nq": 1, "page": 32, "lo": 65571, "hi": 131072, "weights": False},
        # caches grown past their budget by one page or more of new tokens
        {"name": "evict after some tokens", "op": "evict", "B": 16, "Hkv": 8, "D": 128,
         "page": 16, "lo": 1030, "hi": 1152, "budget": 1024, "sink": 4, "recent": 255},
        # long prompts cut down to what was attended to
        {"name": "evict after long prompts", "op": "evict", "B": 4, "Hkv": 8, "D": 128,
         "page": 64, "lo": 20011, "hi": 32768, "budget": 8192, "sink": 4, "recent": 1024},
        # two short prompts of different lengths, padded to one batch
        {"name": "diff prompt short", "op": "diff_prompt", "B": 2, "Hq": 8, "Hkv": 4, "Sq": 333,
         "Skv": 333, "causal": True, "ragged": True, "norm": True, "layer": 3},
        # a long prompt
        {"name": "diff prompt long", "op": "diff_prompt", "B": 1, "Hq": 16, "Hkv": 16, "Sq": 8192,
         "Skv": 8192, "causal": True, "ragged": False, "norm": True, "layer": 12},
        # the next piece of a long document against what came before it
        {"name": "diff prompt piece of a long one", "op": "diff_prompt", "B": 1, "Hq": 16,
         "Hkv": 4, "Sq": 500, "Skv": 32500, "causal": True, "ragged": False, "norm": True,
         "layer": 12},
        # one short conversation: latency
        {"name": "diff decode one sequence", "op": "diff_decode", "B": 1, "Hq": 16, "Hkv": 4,
         "nq": 1, "page": 16, "lo": 1501, "hi": 1501, "norm": True, "layer": 0},
        # an ordinary batch of conversations
        {"name": "diff decode batch", "op": "diff_decode", "B": 16, "Hq": 16, "Hkv": 4, "nq": 1,
         "page": 32, "lo": 1000, "hi": 16001, "norm": True, "layer": 20},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "evict", "diff_prompt", "diff_decode"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        D = rng.choice([64, 128, 256])
        B = _log(rng, 1, 64)
        n = _log(rng, 1, 16000 // B)
        lo = n + rng.randrange(0, 500)
        return {"op": op, "B": B, "n": n, "Hkv": rng.choice([1, 2, 4, 5, 8]), "D": D, "page": page,
                "lo": lo, "hi": lo + rng.randrange(0, 2000), "ragged": rng.random() < 0.5,
                "weights": rng.random() < 0.5}
    if op == "decode":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(40, 500000 // (B * Hkv)))
        return {"op": op, "B": B, "Hq": Hkv * rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16]),
                "Hkv": Hkv, "D": D, "nq": rng.choice([1, 1, 1, 2, 3, 5]), "page": page,
                "lo": rng.randrange(0, hi + 1), "hi": hi, "weights": rng.random() < 0.5}
    if op == "evict":
        Hkv = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 32)
        hi = _log(rng, 20, 500000 // (B * Hkv))
        budget = rng.randrange(1, hi + 1)
        sink = rng.randrange(0, min(budget, 16) + 1)
        return {"op": op, "B": B, "Hkv": Hkv, "D": rng.choice([64, 128, 256]), "page": page,
                "lo": rng.randrange(0, hi + 1), "hi": hi, "budget": budget, "sink": sink,
                "recent": rng.randrange(0, budget - sink + 1)}
    Hkv = rng.choice([1, 2, 3, 4, 8])
    grp = rng.choice([1, 2, 3, 4])
    layer = rng.randrange(0, 32)
    if op == "diff_decode":
        B = _log(rng, 1, 32)
        hi = _log(rng, 1, 250000 // (B * Hkv))
        return {"op": op, "B": B, "Hq": Hkv * grp, "Hkv": Hkv, "nq": rng.choice([1, 1, 1, 2, 4]),
                "page": page, "lo": rng.randrange(0, hi + 1), "hi": hi,
                "norm": rng.random() < 0.7, "layer": layer}
    Sq = _log(rng, 1, 2500)
    Skv = Sq + (0 if rng.random() < 0.5 else _log(rng, 1, 5000))
    return {"op": op, "B": rng.choice([1, 1, 2]), "Hq": Hkv * grp if Hkv < 8 else 8, "Hkv": Hkv,
            "Sq": Sq, "Skv": Skv, "causal": rng.random() < 0.8, "ragged": rng.random() < 0.5,
            "norm": rng.random() < 0.7, "layer": layer}


# ---------------------------------------------------------------- inputs

def _spread(B, lo, hi):
    """B lengths between lo and hi, the longest first, the others scattered."""
    return [hi] + [lo + (hi - lo) * (b * 40503 % 65536) // 65536 for b in range(1, B)]


def _case_lens(case):
    """Cached tokens of every sequence (the new ones included)."""
    return _spread(case["B"], case["lo"], case["hi"])


def _ragged_lens(case):
    """(query lengths, key lengths) of a prompt case."""
    if not case["ragged"]:
        return [case["Sq"]] * case["B"], [case["Skv"]] * case["B"]
    ql = _spread(case["B"], (case["Sq"] + 1) // 2, case["Sq"])
    return ql, [n + case["Skv"] - case["Sq"] for n in ql]


def _new_lens(case):
    if not case["ragged"]:
        return [case["n"]] * case["B"]
    return _spread(case["B"], case["n"] // 2, case["n"])


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pool(case, g, lens, extra=0):
    """A pool with every sequence's pages scattered over it, and `extra` pages for each besides:
    (k_pages, v_pages, table, extra_table)."""
    page, Hkv, D, B = case["page"], case["Hkv"], case.get("D", 128), case["B"]
    counts = [-(-n // page) for n in lens]
    width = max(1, max(counts))
    P = sum(counts) + extra * B + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    first = _i32([sum(counts[:b]) for b in range(B)])[:, None]
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None, :]
    used = col < _i32(counts)[:, None]
    table = torch.where(used, order[(first + col).clamp(max=P - 1).long()], 0).contiguous()
    more = order[sum(counts):sum(counts) + extra * B].reshape(B, extra).contiguous()
    k = torch.randn((P, page, Hkv, D), generator=g, device="cuda", dtype=torch.float16)
    v = torch.randn((P, page, Hkv, D), generator=g, device="cuda", dtype=torch.float16)
    return k, v, table, more


def _lambda_init(layer):
    """The initial lambda of a differential layer by its depth."""
    return 0.8 - 0.6 * math.exp(-0.3 * layer)


def _weights(g, k):
    """Accumulated weights as after a few hundred steps: most tokens hold little, a few much."""
    P, page, Hkv, _ = k.shape
    return torch.randn((P, Hkv, page), generator=g, device="cuda").mul_(1.5).exp_()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]

    def half(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).half()

    if op == "diff_prompt":
        B, Sq, Skv, D = case["B"], case["Sq"], case["Skv"], 128
        # token-major projections, as a model's linear layers leave them; a trained model's
        # scores spread wider than those of unit vectors
        s["q"] = half(B, Sq, case["Hq"], D, std=1.6).permute(0, 2, 1, 3)
        s["k"] = half(B, Skv, case["Hkv"], D).permute(0, 2, 1, 3)
        s["v"] = half(B, Skv, case["Hkv"], D).permute(0, 2, 1, 3)
        ql, kl = _ragged_lens(case)
        s["q_lens"], s["kv_lens"] = (_i32(ql), _i32(kl)) if case["ragged"] else (None, None)
    else:
        lens = _case_lens(case)
        s["lens"] = lens
        s["kv_lens"] = _i32(lens)
        extra = -(-case["budget"] // case["page"]) if op == "evict" else 0
        s["k_pages"], s["v_pages"], s["table"], s["dst_table"] = _pool(case, g, lens, extra)
        D = s["k_pages"].shape[3]
        if op == "append":
            s["k_new"] = half(case["B"], case["n"], case["Hkv"], D).permute(0, 2, 1, 3)
            s["v_new"] = half(case["B"], case["n"], case["Hkv"], D).permute(0, 2, 1, 3)
            s["new_lens"] = _i32(_new_lens(case)) if case["ragged"] else None
        elif op != "evict":
            s["q"] = half(case["B"], case["Hq"], case["nq"], D, std=1.6)
        s["weights"] = _weights(g, s["k_pages"]) if op == "evict" or case.get("weights") else None
    if op.startswith("diff"):
        s["lambda_vecs"] = torch.randn((4, case["Hq"], 64), generator=g, device="cuda").mul_(0.1)
        s["lambda_init"] = _lambda_init(case["layer"])
        s["norm_weight"] = (1 + 0.1 * torch.randn(128, generator=g, device="cuda")
                            if case["norm"] else None)
    return s


def _workspace(gb, s):
    """The scratch that a program keeps for its calls."""
    op = s["op"]
    if op in ("append", "evict"):
        return None
    if op == "decode":
        n = gb.attn_paged_decode_f16_workspace_size(s["B"], s["Hq"], s["Hkv"], s["nq"], s["hi"],
                                                    s["D"], s["weights"] is not None)
    elif op == "diff_decode":
        n = gb.attn_diff_paged_decode_f16_workspace_size(s["B"], s["Hq"], s["Hkv"], s["nq"],
                                                         s["hi"], 128)
    else:
        n = gb.attn_diff_prefill_workspace_size(s["B"], s["Hq"], s["Sq"], s["Skv"], 128)
    return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- the operators

def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "decode": _plain_decode, "evict": _plain_evict,
            "diff_prompt": _plain_diff_prompt, "diff_decode": _plain_diff_decode}[s["op"]](s)


def _run_own(s):
    import attention_fp16_flashattention_gb300 as gb
    if "workspace" not in s:
        s["workspace"] = _workspace(gb, s)
    op, ws = s["op"], s["workspace"]
    if op == "append":
        gb.kv_paged_append_f16(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"],
                               s["kv_lens"], new_lens=s["new_lens"], weights=s["weights"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"]}
    if op == "evict":
        new_lens, kept = gb.kv_paged_evict(s["k_pages"], s["v_pages"], s["weights"], s["table"],
                                           s["kv_lens"], s["budget"], sink=s["sink"],
                                           recent=s["recent"], dst_table=s["dst_table"],
                                           max_kv_len=s["hi"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"],
                "new_lens": new_lens, "kept": kept}
    if op == "decode":
        lse = torch.empty(s["q"].shape[:3], device="cuda")
        o = gb.attn_paged_decode_f16_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"],
                                         s["kv_lens"], max_kv_len=s["hi"], lse=lse,
                                         weights=s["weights"], workspace=ws)
        return {"o": o, "lse": lse, "weights": s["weights"]}
    B, Hq, n, _ = s["q"].shape
    lse = torch.empty((B, Hq, 2, n), device="cuda")
    if op == "diff_decode":
        o = gb.attn_diff_paged_decode_f16_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"],
                                              s["kv_lens"], s["lambda_vecs"], s["lambda_init"],
                                              norm_weight=s["norm_weight"], eps=EPS,
                                              max_kv_len=s["hi"], lse=lse, workspace=ws)
    else:
        o = gb.attn_diff_prefill_fwd(s["q"], s["k"], s["v"], s["lambda_vecs"], s["lambda_init"],
                                     norm_weight=s["norm_weight"], eps=EPS, causal=s["causal"],
                                     q_lens=s["q_lens"], kv_lens=s["kv_lens"], lse=lse,
                                     workspace=ws)
    return {"o": o, "lse": lse}


def _slots(table, page, n):
    """Pool slots (page * size + offset) of logical tokens 0..n-1 of every sequence, [B][n]."""
    t = torch.arange(n, device="cuda")
    return table[:, t // page].long() * page + t % page


def _gather(pages, slots, live):
    """FP32 [B][Hkv][n][D] of the cached rows; rows that are not live hold zeros."""
    P, page, Hkv, D = pages.shape
    rows = pages.reshape(P * page, Hkv, D)[slots].float()
    return torch.where(live[:, :, None, None], rows, 0.0).transpose(1, 2)


def _weight_index(slots, Hkv, page):
    """Flat indexes into weights [P][Hkv][page] of pool slots [B][n]: [B][Hkv][n]."""
    h = torch.arange(Hkv, device="cuda")[None, :, None]
    return ((slots // page)[:, None, :] * Hkv + h) * page + (slots % page)[:, None, :]


def _softmax(x):
    """(probabilities, natural-log sum of exponentials) over the last dimension; a row whose
    scores are all -inf has probabilities 0 and the logarithm -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(-1)
    return p / torch.where(total == 0, 1.0, total), lse


def _plain_append(s):
    B, Hkv, n, D = s["k_new"].shape
    P, page = s["k_pages"].shape[:2]
    count = s["new_lens"] if s["new_lens"] is not None else torch.full_like(s["kv_lens"], n)
    i = torch.arange(n, device="cuda")[None, :]
    live = i < count[:, None]
    tok = ((s["kv_lens"] - count)[:, None] + i).clamp(min=0)
    tok = torch.where(live, tok, 0)
    slots = torch.gather(s["table"].long(), 1, tok // page) * page + tok % page
    to = slots[live]
    s["k_pages"].view(P * page, Hkv, D)[to] = s["k_new"].transpose(1, 2)[live]
    s["v_pages"].view(P * page, Hkv, D)[to] = s["v_new"].transpose(1, 2)[live]
    if s["weights"] is not None:
        h = torch.arange(Hkv, device="cuda")[None, :]
        s["weights"][(to // page)[:, None], h, (to % page)[:, None]] = 0.0
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"]}


def _visible(s, n):
    """[B][1][nq][n]: whether query i of a sequence sees cached token t."""
    t = torch.arange(n, device="cuda")
    pos = s["kv_lens"][:, None] - s["nq"] + torch.arange(s["nq"], device="cuda")
    return t[None, None, None, :] <= pos[:, None, :, None]


def _plain_decode(s):
    B, Hq, nq, D = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    grp, n = Hq // Hkv, s["hi"]
    slots = _slots(s["table"], page, n)
    live = torch.arange(n, device="cuda")[None, :] < s["kv_lens"][:, None]
    k, v = _gather(s["k_pages"], slots, live), _gather(s["v_pages"], slots, live)
    q = s["q"].float().reshape(B, Hkv, grp * nq, D)
    x = (q @ k.transpose(2, 3)).reshape(B, Hq, nq, n) * (1 / math.sqrt(D))
    p, lse = _softmax(torch.where(_visible(s, n), x, -math.inf))
    p = p.reshape(B, Hkv, grp * nq, n)
    o = (p @ v).reshape(B, Hq, nq, D).half()
    if s["weights"] is not None:
        at = _weight_index(slots, Hkv, page)[live[:, None, :].expand(B, Hkv, n)]
        got = p.sum(2)[live[:, None, :].expand(B, Hkv, n)]
        s["weights"].view(-1)[at] += got
    return {"o": o, "lse": lse, "weights": s["weights"]}


def _plain_evict(s):
    P, page, Hkv, D = s["k_pages"].shape
    B, n, budget = s["B"], s["hi"], s["budget"]
    lens = s["kv_lens"].long()
    slots = _slots(s["table"], page, n)
    at = _weight_index(slots, Hkv, page)
    w = s["weights"].view(-1)[at]                                     # [B][Hkv][n]
    t = torch.arange(n, device="cuda")
    held = (t[None, :] < s["sink"]) | (t[None, :] >= lens[:, None] - s["recent"])
    rank = torch.where(held[:, None, :], math.inf, w)
    rank = torch.where((t[None, :] < lens[:, None])[:, None, :], rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = order[:, :, :min(budget, n)].sort(-1).values               # [B][Hkv][kept]
    new_lens = lens.clamp(max=budget)
    m = kept.shape[2]
    j = torch.arange(m, device="cuda")
    # a sequence within its budget keeps everything where it is
    moves = (lens > budget)[:, None, None] & (j < new_lens[:, None])[:, None, :].expand(B, Hkv, m)
    src = torch.gather(slots[:, None, :].expand(B, Hkv, n), 2, kept)
    dst_slots = _slots(s["dst_table"], page, m)[:, None, :].expand(B, Hkv, m)
    stay = (lens <= budget)[:, None, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None].expand(B, Hkv, m)
    # and moves to the new pages all the same
    moves = moves | (stay & (j < new_lens[:, None])[:, None, :])
    src, dst_slots, h = src[moves], dst_slots[moves], h[moves]
    for name in ("k_pages", "v_pages"):
        rows = s[name].view(P * page, Hkv, D)
        rows[dst_slots, h] = rows[src, h]
    values = s["weights"][src // page, h, src % page]
    s["weights"][dst_slots // page, h, dst_slots % page] = values
    out = torch.full((B, Hkv, budget), -1, dtype=torch.int32, device="cuda")
    out[:, :, :m] = torch.where((j < new_lens[:, None])[:, None, :], kept, -1).int()
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"],
            "new_lens": new_lens.int(), "kept": out}


def _lambda(s):
    """The factor of the second map for every query head: FP32 [Hq]."""
    q1, k1, q2, k2 = s["lambda_vecs"].unbind(0)
    return torch.exp((q1 * k1).sum(-1)) - torch.exp((q2 * k2).sum(-1)) + s["lambda_init"]


def _combine(s, p1, p2, v, shape):
    """(p1 - lambda p2) v for [B][Hkv][grp][n][keys] maps, normalised over the head width."""
    Hkv = s["Hkv"]
    lam = _lambda(s).reshape(1, Hkv, -1, 1, 1)
    o = (p1 - lam * p2) @ v[:, :, None]
    if s["norm_weight"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS)
        o = o * s["norm_weight"] * (1 - s["lambda_init"])
    return o.reshape(shape).half()


def _diff(s, q, k, v, visible):
    """Differential attention of q [B][Hq][n][D] with k, v [B][Hkv][keys][D], all FP32;
    visible [B][n][keys]."""
    B, Hq, n, D = q.shape
    d = D // 2
    q = q.reshape(B, s["Hkv"], -1, n, D)
    see = visible[:, None, None]
    x1 = (q[..., :d] @ k[:, :, None, :, :d].transpose(3, 4)) * (1 / math.sqrt(d))
    p1, lse1 = _softmax(torch.where(see, x1, -math.inf))
    del x1
    x2 = (q[..., d:] @ k[:, :, None, :, d:].transpose(3, 4)) * (1 / math.sqrt(d))
    p2, lse2 = _softmax(torch.where(see, x2, -math.inf))
    del x2
    lse = torch.stack([lse1.reshape(B, Hq, n), lse2.reshape(B, Hq, n)], 2)
    return {"o": _combine(s, p1, p2, v, (B, Hq, n, D)), "lse": lse}


def _plain_diff_decode(s):
    n = s["hi"]
    slots = _slots(s["table"], s["page"], n)
    live = torch.arange(n, device="cuda")[None, :] < s["kv_lens"][:, None]
    k, v = _gather(s["k_pages"], slots, live), _gather(s["v_pages"], slots, live)
    return _diff(s, s["q"].float(), k, v, _visible(s, n)[:, 0])


def _plain_diff_prompt(s):
    B, Hq, Sq, D = s["q"].shape
    Skv = s["Skv"]
    ql = s["q_lens"] if s["q_lens"] is not None else torch.full((B,), Sq, device="cuda")
    kl = s["kv_lens"] if s["kv_lens"] is not None else torch.full((B,), Skv, device="cuda")
    i = torch.arange(Sq, device="cuda")[None, :, None]
    t = torch.arange(Skv, device="cuda")[None, None, :]
    see = (t < kl[:, None, None]) & (i < ql[:, None, None])
    if s["causal"]:
        see = see & (t <= i + (kl - ql)[:, None, None])
    v = torch.where((t[0, 0] < kl[:, None])[:, None, :, None], s["v"].float(), 0.0)
    return _diff(s, s["q"].float(), s["k"].float(), v, see)


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(ql, kl, causal):
    """Visible (query, key) pairs of one sequence."""
    if not causal:
        return ql * kl
    first = kl - ql + 1                         # keys that query 0 sees
    short = max(0, min(ql, 1 - first))          # queries that see none
    return (ql - short) * (max(first, 1) + kl) // 2


def work(case):
    op, B = case["op"], case["B"]
    if op == "diff_prompt":
        Hq, D = case["Hq"], 128
        ql, kl = _ragged_lens(case)
        pairs = sum(_pairs(a, b, case["causal"]) for a, b in zip(ql, kl))
        rows = 2 * D * (2 * Hq * B * case["Sq"] + 2 * case["Hkv"] * sum(kl))
        return {"bytes": rows + 8 * Hq * B * case["Sq"],
                "flops": 2 * Hq * pairs * (2 * (D // 2) + 2 * D)}
    lens, D, Hkv = _case_lens(case), case.get("D", 128), case["Hkv"]
    if op == "append":
        new = sum(_new_lens(case))
        return {"bytes": new * Hkv * (8 * D + (4 if case["weights"] else 0)), "flops": 0}
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": Hkv * (kept * (8 * D + 8) + 4 * sum(lens)), "flops": 0}
    maps = 2 if op == "diff_decode" else 1
    rows = B * case["Hq"] * case["nq"]
    tokens = sum(lens)
    weights = 8 * Hkv * tokens if case.get("weights") else 0
    qk = 2 * D if op == "decode" else 2 * (D // 2) * maps
    return {"bytes": 4 * D * Hkv * tokens + rows * (4 * D + 4 * maps) + weights,
            "flops": case["Hq"] * case["nq"] * tokens * (qk + 2 * D * maps)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "decode": _exact_decode, "evict": _exact_evict,
                "diff_prompt": _exact_diff_prompt, "diff_decode": _exact_diff_decode}[s["op"]](s)


def _sequence(s, pages, b, n):
    """The first n cached rows of sequence b: float64 [n][Hkv][D]."""
    P, page, Hkv, D = pages.shape
    used = s["table"][b, :-(-n // page)].long()
    return pages[used].reshape(-1, Hkv, D)[:n].double()


def _rows_of(scores):
    """(normalised exponentials, logarithms of their sums) of rows of float64 scores."""
    lse = torch.logsumexp(scores, -1)
    return torch.exp(scores - lse[:, None]), lse


def _exact_append(s):
    page = s["page"]
    table = s["table"].tolist()
    for b, (n, new) in enumerate(zip(s["lens"], _new_lens(s))):
        lo = n - new
        for p in range(lo // page, -(-n // page)):
            a, z = max(lo, p * page), min(n, (p + 1) * page)
            if z <= a:
                continue
            to, at = table[b][p], slice(a - p * page, z - p * page)
            s["k_pages"][to, at] = s["k_new"][b, :, a - lo:z - lo].transpose(0, 1)
            s["v_pages"][to, at] = s["v_new"][b, :, a - lo:z - lo].transpose(0, 1)
            if s["weights"] is not None:
                s["weights"][to, :, at] = 0
    w = s["weights"]
    return {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(),
            "weights": None if w is None else w.double()}


def _exact_decode(s):
    B, Hq, nq, D = s["q"].shape
    grp, page = Hq // s["Hkv"], s["page"]
    o = torch.zeros((B, Hq, nq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    w = None if s["weights"] is None else s["weights"].double()
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        k, v = _sequence(s, s["k_pages"], b, n), _sequence(s, s["v_pages"], b, n)
        for h in range(s["Hkv"]):
            got = torch.zeros(n, dtype=torch.float64, device="cuda")
            for i in range(nq):
                m = n - nq + i + 1                          # tokens that query i sees
                if m <= 0:
                    continue
                heads = slice(h * grp, (h + 1) * grp)
                x = s["q"][b, heads, i].double() @ k[:m, h].T / math.sqrt(D)
                p, lse[b, heads, i] = _rows_of(x)
                o[b, heads, i] = p @ v[:m, h]
                got[:m] += p.sum(0)
            if w is not None:
                t = torch.arange(n, device="cuda")
                w[s["table"][b].long()[t // page], h, t % page] += got
    return {"o": o, "lse": lse, "weights": w}


def _exact_evict(s):
    page, budget, Hkv = s["page"], s["budget"], s["Hkv"]
    kept = torch.full((s["B"], Hkv, budget), -1, dtype=torch.int64, device="cuda")
    k, v, w = s["k_pages"].double(), s["v_pages"].double(), s["weights"].double()
    for b, n in enumerate(s["lens"]):
        t = torch.arange(n, device="cuda")
        src = s["table"][b].long()[t // page], t % page
        lo, hi = s["sink"], max(s["sink"], n - s["recent"])
        for h in range(Hkv):
            keep = t
            if n > budget:
                middle = s["weights"][src[0][lo:hi], h, src[1][lo:hi]]
                count = budget - lo - (n - hi)
                best = torch.argsort(middle, descending=True, stable=True)[:count] + lo
                keep = torch.cat([t[:lo], torch.sort(best).values, t[hi:]])
            m = keep.numel()
            kept[b, h, :m] = keep
            j = torch.arange(m, device="cuda")
            to = s["dst_table"][b].long()[j // page], j % page
            at = src[0][keep], src[1][keep]
            k[to[0], to[1], h] = s["k_pages"][at[0], at[1], h].double()
            v[to[0], to[1], h] = s["v_pages"][at[0], at[1], h].double()
            w[to[0], h, to[1]] = s["weights"][at[0], h, at[1]].double()
    new_lens = torch.tensor([min(n, budget) for n in s["lens"]], device="cuda")
    return {"k_pages": k, "v_pages": v, "weights": w, "new_lens": new_lens, "kept": kept}


def _exact_diff_head(s, q, k, v, h):
    """One head: q [n][D], k, v [keys][D] float64, first[i] = keys that row i sees."""
    d = q.shape[-1] // 2
    vec = s["lambda_vecs"][:, h].double()
    lam = math.exp(float(vec[0] @ vec[1])) - math.exp(float(vec[2] @ vec[3])) + s["lambda_init"]
    outs, sums = [], []
    for part in (slice(0, d), slice(d, 2 * d)):
        p, lse = _rows_of(q[:, part] @ k[:, part].T / math.sqrt(d) + s["bias"])
        outs.append(p @ v)
        sums.append(lse)
    o = outs[0] - lam * outs[1]
    if s["norm_weight"] is not None:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS)
        o = o * s["norm_weight"].double() * (1 - s["lambda_init"])
    return o, torch.stack(sums)


def _exact_diff(s, b, q, k, v, first, o, lse):
    """All heads of sequence b: row i of q [Hq][n][D] sees the keys before first + i (or all)."""
    Hq, n, _ = q.shape
    keys, grp = k.shape[0], Hq // s["Hkv"]
    i, t = torch.arange(n, device="cuda"), torch.arange(keys, device="cuda")
    skip = 0
    s["bias"] = torch.zeros((), dtype=torch.float64, device="cuda")
    if first is not None:
        skip = min(n, max(0, 1 - first))                     # rows that see nothing
        see = t[None, :] < first + i[skip:, None]
        s["bias"] = torch.where(see, 0.0, -math.inf).double()
    if skip == n or keys == 0:
        return
    for h in range(Hq):
        hk = h // grp
        o[b, h, skip:n], lse[b, h, :, skip:n] = _exact_diff_head(
            s, q[h, skip:].double(), k[:, hk].double(), v[:, hk].double(), h)


def _exact_diff_out(s):
    B, Hq, n, D = s["q"].shape
    o = torch.zeros((B, Hq, n, D), dtype=torch.float64, device="cuda")
    return o, torch.full((B, Hq, 2, n), -math.inf, dtype=torch.float64, device="cuda")


def _exact_diff_decode(s):
    o, lse = _exact_diff_out(s)
    for b, n in enumerate(s["lens"]):
        _exact_diff(s, b, s["q"][b], _sequence(s, s["k_pages"], b, n),
                    _sequence(s, s["v_pages"], b, n), n - s["nq"] + 1, o, lse)
    return {"o": o, "lse": lse}


def _exact_diff_prompt(s):
    o, lse = _exact_diff_out(s)
    ql, kl = _ragged_lens(s)
    for b in range(s["B"]):
        _exact_diff(s, b, s["q"][b, :, :ql[b]], s["k"][b, :, :kl[b]].transpose(0, 1),
                    s["v"][b, :, :kl[b]].transpose(0, 1), kl[b] - ql[b] + 1 if s["causal"] else None,
                    o, lse)
    return {"o": o, "lse": lse}
