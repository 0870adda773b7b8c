"""What a serving step needs around the paged caches: page tables and slot maps, norms and rotary
positions of queries and keys (also on their way into the cache), and decode of requests that share a
prefix; what is measured of them, and their plain forms.

`run` computes one pass of an operator from `prepare`'s state: with elementary torch operations
in FP32 (angles in FP64), or, where `own` is true, by the library's calls.  `exact` is the definition
in float64.

A cache is a pool of pages k_pages, v_pages [P][page][Hkv][D] (FP16, or E4M3 bytes with a scale) with
one page-table row per sequence; the pages that no sequence holds are on a stack, free_pages and
free_count.  A slot is page * page_size + offset.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a busy server: a slot for one token of each of 64 sequences
        {"name": "extend one token", "op": "extend", "B": 64, "lo": 300, "hi": 6000, "new_lo": 1,
         "new_hi": 1, "page": 16},
        # 32 new requests: pages and slots of their whole prompts
        {"name": "extend prompts", "op": "extend", "B": 32, "lo": 0, "hi": 0, "new_lo": 501,
         "new_hi": 8192, "page": 64},
        # drafted tokens that were not accepted
        {"name": "release drafts", "op": "release", "B": 64, "lo": 300, "hi": 6000, "drop": 24,
         "page": 16},
        # long documents end
        {"name": "release long documents", "op": "release", "B": 16, "lo": 65571, "hi": 131072,
         "drop": None, "page": 16},
        # two short prompts, adjacent pairs in half of the head
        {"name": "rotate short prompts", "op": "rope", "B": 2, "S": 333, "Hq": 8, "Hkv": 4, "D": 64,
         "rot": 32, "axes": 1, "interleaved": True, "norm": False, "far": 0},
        # queries and keys of the benchmark's video attention: three axes of positions, norms
        {"name": "rotate video tokens", "op": "rope", "B": 1, "S": 32768, "Hq": 24, "Hkv": 24,
         "D": 128, "rot": 128, "axes": 3, "interleaved": False, "norm": True, "far": 0},
        # one decoding step of a busy server
        {"name": "rotate and append one token", "op": "append", "B": 64, "lo": 1, "hi": 1, "Hq": 32,
         "Hkv": 8, "D": 128, "rot": 128, "interleaved": False, "norm": True, "page": 16,
         "e4m3": False, "far": 6000},
        # prompts of eight requests end to end, two norms
        {"name": "rotate and append prompts", "op": "append", "B": 8, "lo": 700, "hi": 4001,
         "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "interleaved": False, "norm": True, "page": 64,
         "e4m3": False, "far": 0},
        # the next piece of a long document into an E4M3 cache: the benchmark's heads, a quarter of
        # the head rotated, positions past what the model was trained on
        {"name": "rotate and append E4M3", "op": "append", "B": 1, "lo": 8192, "hi": 8192, "Hq": 6,
         "Hkv": 1, "D": 256, "rot": 64, "interleaved": False, "norm": False, "page": 32,
         "e4m3": True, "far": 122880},
        # a few requests behind a short instruction: latency
        {"name": "shared short prefix", "op": "shared", "groups": "8x1024", "Hq": 32, "Hkv": 8,
         "D": 128, "nq": 1, "page": 16, "lo": 1, "hi": 300},
        # a busy server, every request behind the same long instruction
        {"name": "shared long prefix", "op": "shared", "groups": "64x16384", "Hq": 32, "Hkv": 8,
         "D": 128, "nq": 1, "page": 64, "lo": 100, "hi": 2001},
        # questions on several long documents, some requests with none; the benchmark's heads
        {"name": "shared documents", "op": "shared", "groups": "12x65536 1x0 5x98304 7x32768 1x0",
         "Hq": 6, "Hkv": 1, "D": 256, "nq": 2, "page": 32, "lo": 37, "hi": 3001},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "release", "rope", "append", "append", "shared", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "extend":
        B = _log(rng, 1, 512)
        new = _log(rng, 1, max(2, 120000 // B))
        lo = rng.randrange(0, 3000)
        return {"op": op, "B": B, "lo": lo, "hi": lo + rng.randrange(0, 3000),
                "new_lo": rng.randrange(0, new + 1), "new_hi": new, "page": page}
    if op == "release":
        B = _log(rng, 1, 512)
        hi = _log(rng, 1, max(2, 1000000 // B))
        return {"op": op, "B": B, "lo": rng.randrange(0, hi + 1), "hi": hi,
                "drop": None if rng.random() < 0.5 else _log(rng, 1, 300), "page": page}
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 8])
    rot = rng.choice([D, D, D, D // 2, D // 4])
    if op == "rope":
        B = rng.choice([1, 1, 2, 5])
        return {"op": op, "B": B, "S": _log(rng, 1, 400000 // (B * (Hq + Hkv))), "Hq": Hq,
                "Hkv": Hkv, "D": D, "rot": rot, "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6,
                "far": rng.choice([0, 5000, 1000000])}
    if op == "append":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, 300000 // (B * (Hq + 2 * Hkv))))
        return {"op": op, "B": B, "lo": rng.randrange(1, hi + 1), "hi": hi, "Hq": Hq, "Hkv": Hkv,
                "D": D, "rot": rot, "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6,
                "page": page, "e4m3": rng.random() < 0.4, "far": rng.choice([0, 5000, 200000])}
    n = rng.choice([1, 1, 2, 3, 6])
    nq = rng.choice([1, 1, 1, 2, 4])
    groups = []
    for _ in range(n):
        members = _log(rng, 1, 48 // n)
        cap = min(200000 // (n * Hkv), 18000000 // (n * members * Hq * nq))
        groups.append((members, page * rng.randrange(0, max(1, _log(rng, 256, cap) // page) + 1)))
    members = sum(m for m, _ in groups)
    hi = _log(rng, nq, max(nq + 1, 100000 // (members * Hkv)))
    return {"op": op, "groups": " ".join("%dx%d" % g for g in groups), "Hq": Hq, "Hkv": Hkv,
            "D": D, "nq": nq, "page": page, "lo": rng.randrange(0, hi + 1), "hi": hi}


# ---------------------------------------------------------------- inputs

def _spread(B, lo, hi):
    """B lengths between lo and hi, the longest first, the others scattered."""
    return [hi] + [lo + (hi - lo) * (b * 40503 % 65536) // 65536 for b in range(1, B)]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cases_lens(case):
    """What is known on the host of a table case: (cached, new or kept) tokens per sequence."""
    lens = _spread(case["B"], case["lo"], case["hi"])
    if case["op"] == "extend":
        new = _spread(case["B"], case["new_lo"], case["new_hi"])
        return lens, new
    if case["drop"] is None:
        return lens, [0] * case["B"]
    return lens, [max(0, n - 1 - case["drop"] * (b * 40503 % 65536) // 65536)
                  for b, n in enumerate(lens)]


def _groups(case):
    """(sequences, tokens that they share) of every group of a case's "8x1024 1x0"."""
    return [tuple(int(n) for n in g.split("x")) for g in case["groups"].split()]


def _pages(n, page):
    return -(-n // page)


def _frequencies(case):
    """Angles per position, FP32 [rot / 2], of one axis after the other; far positions use
    frequencies stretched for a long context: the slow ones divided, the fast ones kept."""
    rot, axes = case["rot"], case.get("axes", 1)
    out = []
    for n in _sections(rot, axes):
        f = 10000.0 ** (-np.arange(n, dtype=np.float64) / n)
        if case["far"] > 10000:
            turns = 8192 * f / (2 * math.pi)
            keep = np.clip((turns - 1) / 31, 0, 1)
            f = f * (keep + (1 - keep) / 16)
        out.append(f)
    return torch.from_numpy(np.concatenate(out).astype(np.float32)).cuda()


def _sections(rot, axes):
    """Pairs of each axis of positions, the first axis with what is left over."""
    rest = [rot // 2 // 4 if axes == 3 else rot // 2 // 2] * (axes - 1)
    return [rot // 2 - sum(rest)] + rest


def _rope_scale(case):
    return 1.0 + 0.1 * math.log(16) if case["far"] > 10000 else 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op, page = case["op"], case.get("page")

    def half(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).half()

    def pool(P, Hkv, D, e4m3=False):
        if e4m3:
            return [torch.randint(0, 120, (P, page, Hkv, D), generator=g, device="cuda",
                                  dtype=torch.uint8) for _ in range(2)]
        return [torch.randn((P, page, Hkv, D), generator=g, device="cuda", dtype=torch.float16)
                for _ in range(2)]

    if op in ("extend", "release"):
        lens, other = _cases_lens(case)
        after = [a + b for a, b in zip(lens, other)] if op == "extend" else lens
        held = sum(_pages(n, page) for n in lens)
        P = sum(_pages(n, page) for n in after) + 37
        width = max(1, max(_pages(n, page) for n in after)) + 2
        order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        s["page_table"] = _table(order, lens, page, width)
        free = torch.cat([order[held:], order[:held]])   # the stack; what lies above it is stale
        s.update(P=P, kv_lens=_i32(lens), free_pages=free.contiguous(), free_count=_i32([P - held]))
        s["new_lens" if op == "extend" else "keep_lens"] = _i32(other)
        s["tokens"] = sum(other)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "shared":
        return _prepare_shared(case, s, g, half, pool)
    s["freqs"] = _frequencies(case)
    s["rope_scale"] = _rope_scale(case)
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        s["q_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
        s["k_weight"] = 1 + 0.2 * torch.randn(D, generator=g, device="cuda")
    if op == "rope":
        B, S, axes = case["B"], case["S"], case["axes"]
        # token-major projections packed as a model's linear layer leaves them
        qkv = half(B, S, Hq + Hkv, D, std=1.6)
        s["q"], s["k"] = (x.permute(0, 2, 1, 3) for x in qkv.split([Hq, Hkv], 2))
        t = torch.arange(S, device="cuda", dtype=torch.int32) + case["far"]
        # a grid of 32 x 32 positions in every frame
        grid = [t] if axes == 1 else [t // 32, t % 32] if axes == 2 else \
            [t // 1024, t // 32 % 32, t % 32]
        s["positions"] = torch.stack(grid)[:, None].expand(axes, B, S).contiguous()
        s["sections"] = _sections(case["rot"], axes) if axes > 1 else None
        return s
    lens = _spread(case["B"], case["lo"], case["hi"])
    T = sum(lens)
    s["lens"] = lens
    qkv = half(1, T, Hq + 2 * Hkv, D, std=1.6)
    s["q"], s["k"], s["v"] = (x.permute(0, 2, 1, 3) for x in qkv.split([Hq, Hkv, Hkv], 2))
    before = [(case["far"] + b * 7919) % (case["far"] + 1) for b in range(case["B"])]
    where = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(before, lens)])
    s["positions"] = where.to(torch.int32)[None].contiguous()
    counts = [_pages(a + n, page) - a // page for a, n in zip(before, lens)]
    P = sum(counts) + 5
    order = torch.randperm(P, generator=g, device="cuda")
    slots, at = [], 0
    for a, n, c in zip(before, lens, counts):
        t = torch.arange(a, a + n, device="cuda")
        slots.append(order[at + t // page - a // page] * page + t % page)
        at += c
    s["slots"] = torch.cat(slots).to(torch.int32)[None].contiguous()
    s["k_pages"], s["v_pages"] = pool(P, Hkv, D, case["e4m3"])
    s["k_scale"], s["v_scale"] = (0.0375, 0.021) if case["e4m3"] else (1.0, 1.0)
    return s


def _table(order, lens, page, width):
    """Page-table rows with the pages of `order` given to the sequences one after the other."""
    counts = [_pages(n, page) for n in lens]
    first = _i32([sum(counts[:b]) for b in range(len(lens))])[:, None]
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None, :]
    at = (first + col).clamp(max=order.numel() - 1).long()
    return torch.where(col < _i32(counts)[:, None], order[at], -1).contiguous()


def _prepare_shared(case, s, g, half, pool):
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    groups = _groups(case)
    members = [m for m, _ in groups]
    B, n_groups = sum(members), len(members)
    own_lens = _spread(B, case["lo"], case["hi"])
    prefix_of = [p for m, p in groups for _ in range(m)]
    group_of = [i for i, m in enumerate(members) for _ in range(m)]
    own_pages = [_pages(n, page) for n in own_lens]
    pre_pages = [p // page for _, p in groups]
    P = sum(own_pages) + sum(pre_pages) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    width = max(1, max(p // page + o for p, o in zip(prefix_of, own_pages)))
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    at = sum(pre_pages)
    for b in range(B):
        i = group_of[b]
        start, n = sum(pre_pages[:i]), pre_pages[i]
        table[b, :n] = order[start:start + n]
        table[b, n:n + own_pages[b]] = order[at:at + own_pages[b]]
        at += own_pages[b]
    s.update(B=B, groups=groups, own_lens=own_lens, prefix_of=prefix_of, page_table=table,
             kv_lens=_i32([p + n for p, n in zip(prefix_of, own_lens)]),
             group_starts=_i32([sum(members[:i]) for i in range(n_groups + 1)]),
             prefix_lens=_i32([p for _, p in groups]),
             max_prefix=max(p for _, p in groups))
    s["k_pages"], s["v_pages"] = pool(P, Hkv, D)
    s["q"] = half(B, case["Hq"], case["nq"], D, std=1.6)
    return s


# ---------------------------------------------------------------- the operators

def run(s):
    if own:
        return _run_own(s)
    return {"extend": _plain_extend, "release": _plain_release, "rope": _plain_rope,
            "append": _plain_append, "shared": _plain_shared}[s["op"]](s)


def _run_own(s):
    import attention_fp16_flashattention_gb300 as gb
    op = s["op"]
    if op == "extend":
        lens, count, starts, positions, slots = gb.kv_paged_extend(
            s["page_table"], s["kv_lens"], s["new_lens"], s["free_pages"], s["free_count"],
            s["page"], s["P"], max_tokens=s["tokens"])
        return {"page_table": s["page_table"], "kv_lens": lens, "free_count": count,
                "token_starts": starts, "positions": positions, "slots": slots}
    if op == "release":
        count = gb.kv_paged_release(s["page_table"], s["kv_lens"], s["free_pages"],
                                    s["free_count"], s["page"], s["P"], keep_lens=s["keep_lens"])
        return {"free_pages": s["free_pages"], "free_count": count}
    if op == "rope":
        q, k = gb.qk_norm_rope_f16(s["q"], s["k"], s["positions"], s["freqs"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                   interleaved=s["interleaved"], sections=s["sections"],
                                   rope_scale=s["rope_scale"])
        return {"q": q, "k": k}
    if op == "append":
        q = gb.kv_paged_rope_append(s["q"], s["k"], s["v"], s["slots"], s["k_pages"], s["v_pages"],
                                    s["positions"], s["freqs"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"],
                                    rope_scale=s["rope_scale"], k_scale=s["k_scale"],
                                    v_scale=s["v_scale"])
        return {"q": q, "k_pages": _values(s, "k_pages"), "v_pages": _values(s, "v_pages")}
    if "workspace" not in s:   # the scratch that a program keeps for its calls
        n = gb.attn_paged_decode_shared_f16_workspace_size(
            s["B"], s["Hq"], s["Hkv"], s["nq"], len(s["groups"]), s["max_prefix"], s["hi"], s["D"])
        s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    lse = torch.empty(s["q"].shape[:3], device="cuda")
    o = gb.attn_paged_decode_shared_f16_fwd(s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                            s["kv_lens"], s["group_starts"], s["prefix_lens"],
                                            max_prefix_len=s["max_prefix"], max_own_len=s["hi"],
                                            lse=lse, workspace=s["workspace"])
    return {"o": o, "lse": lse}


def _values(s, name):
    """The pool as the values that it stands for."""
    return s[name].view(torch.float8_e4m3fn) if s.get("e4m3") else s[name]


def _plain_extend(s):
    table, page = s["page_table"], s["page"]
    B, width = table.shape
    old, new, free = s["kv_lens"].long(), s["new_lens"].long(), s["free_count"].long()
    p0 = (old + page - 1) // page
    need = (old + new + page - 1) // page - p0
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= free)
    first = upto - need
    j = torch.arange(width, device="cuda")[None, :] - p0[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & served[:, None]
    at = (free - 1 - first[:, None] - j).clamp(0, s["P"] - 1)
    table.copy_(torch.where(fresh, s["free_pages"][at], table))
    lens = torch.where(served, old + new, old)
    starts = torch.cat([torch.zeros_like(free), new.cumsum(0)])
    T = s["tokens"]
    marks = torch.zeros(T + 1, dtype=torch.int64, device="cuda")
    marks.index_add_(0, starts[1:], torch.ones_like(new))
    b = marks[:T].cumsum(0)                                   # the sequence of every token
    pos = torch.arange(T, device="cuda") - starts[b] + old[b]
    slot = table[b, pos // page].long() * page + pos % page
    return {"page_table": table, "kv_lens": lens.int(),
            "free_count": free.int() - (need * served).sum(0, keepdim=True).int(),
            "token_starts": starts.int(), "positions": torch.where(served[b], pos, -1).int(),
            "slots": torch.where(served[b], slot, -1).int()}


def _plain_release(s):
    table, page = s["page_table"], s["page"]
    width = table.shape[1]
    p0 = (s["keep_lens"].long() + page - 1) // page
    p1 = (s["kv_lens"].long() + page - 1) // page
    count = p1 - p0
    first = count.cumsum(0) - count + s["free_count"].long()
    col = torch.arange(width, device="cuda")[None, :]
    live = (col >= p0[:, None]) & (col < p1[:, None])
    to = first[:, None] + col - p0[:, None]
    # the entries that stay go nowhere: one place behind the list's end
    room = torch.cat([s["free_pages"], torch.zeros_like(s["free_pages"][:1])])
    room[torch.where(live, to, s["P"])] = table
    s["free_pages"].copy_(room[:-1])
    return {"free_pages": s["free_pages"],
            "free_count": (s["free_count"] + count.sum(0, keepdim=True)).int()}


def _plain_rotate(s, x, weight):
    """Norm and rotation of x [B][H][S][D], FP32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    rot = s["rot"]
    pos = s["positions"]
    if s.get("sections"):
        axis = torch.cat([torch.full((n,), i, device="cuda") for i, n in enumerate(s["sections"])])
        pos = pos[axis].permute(1, 2, 0)                       # [B][S][rot / 2]
    else:
        pos = pos.reshape(-1, pos.shape[-1])[:, :, None]
    angle = pos.double() * s["freqs"].double()
    cos = (torch.cos(angle) * s["rope_scale"]).float()[:, None]
    sin = (torch.sin(angle) * s["rope_scale"]).float()[:, None]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    return {"q": _plain_rotate(s, s["q"], s["q_weight"]).half(),
            "k": _plain_rotate(s, s["k"], s["k_weight"]).half()}


def _plain_append(s):
    P, page, Hkv, D = s["k_pages"].shape
    at = s["slots"][0].long()
    for name, x, scale in (("k_pages", _plain_rotate(s, s["k"], s["k_weight"]), s["k_scale"]),
                           ("v_pages", s["v"].float(), s["v_scale"])):
        rows = x[0].transpose(0, 1)                            # [T][Hkv][D]
        if s["e4m3"]:
            code = (rows / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            code = rows.half()
        s[name].view(P * page, Hkv, D)[at] = code
    return {"q": _plain_rotate(s, s["q"], s["q_weight"]).half(), "k_pages": _values(s, "k_pages"),
            "v_pages": _values(s, "v_pages")}


def _rows(pages, table, n):
    """FP32 [...][Hkv][n][D] of the first n cached rows by the page-table rows [...][width]."""
    P, page, Hkv, D = pages.shape
    t = torch.arange(n, device="cuda")
    slots = table[..., t // page].long() * page + t % page
    return pages.reshape(P * page, Hkv, D)[slots].float().transpose(-3, -2)


def _plain_shared(s):
    B, Hq, nq, D = s["q"].shape
    Hkv, page, n = s["Hkv"], s["page"], max(s["hi"], 1)
    grp = Hq // Hkv
    scale = 1 / math.sqrt(D)
    q = s["q"].float().reshape(B, Hkv, grp, nq, D)
    # every sequence's own tokens
    first = _i32([p // page for p in s["prefix_of"]])[:, None]
    col = (torch.arange(_pages(n, page), device="cuda")[None, :] + first)
    table = torch.gather(s["page_table"], 1, col.clamp(max=s["page_table"].shape[1] - 1).long())
    t = torch.arange(n, device="cuda")
    mine = s["kv_lens"] - _i32(s["prefix_of"])
    live = (t[None, :] < mine[:, None])[:, None, :, None]
    k = torch.where(live, _rows(s["k_pages"], table, n), 0.0)
    v = torch.where(live, _rows(s["v_pages"], table, n), 0.0)
    pos = mine[:, None] - nq + torch.arange(nq, device="cuda")
    see = (t <= pos[:, :, None])[:, None, None]
    x = (q.reshape(B, Hkv, grp * nq, D) @ k.transpose(2, 3)).reshape(B, Hkv, grp, nq, n) * scale
    x = torch.where(see, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    # and what its group has in common
    shared, b0 = [], 0
    for members, prefix in s["groups"]:
        b1 = b0 + members
        if prefix:
            kp = _rows(s["k_pages"], s["page_table"][b0], prefix)
            y = q[b0:b1].permute(1, 0, 2, 3, 4).reshape(Hkv, members * grp * nq, D)
            y = (y @ kp.transpose(1, 2)).reshape(Hkv, members, grp, nq, prefix).transpose(0, 1) * scale
            behind = pos[b0:b1, None, None, :, None] + prefix
            y = torch.where(torch.arange(prefix, device="cuda") <= behind, y, -math.inf)
            top[b0:b1] = torch.maximum(top[b0:b1], y.amax(-1, keepdim=True))
            shared.append((b0, b1, prefix, y))
        b0 = b1
    base = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - base)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, Hkv, grp * nq, n) @ v).reshape(B, Hkv, grp, nq, D)
    for b0, b1, prefix, y in shared:
        p = torch.exp(y - base[b0:b1])
        total[b0:b1] += p.sum(-1, keepdim=True)
        vp = _rows(s["v_pages"], s["page_table"][b0], prefix)
        p = p.transpose(0, 1).reshape(Hkv, (b1 - b0) * grp * nq, prefix)
        o[b0:b1] += (p @ vp).reshape(Hkv, b1 - b0, grp, nq, D).transpose(0, 1)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (base + torch.log(total))[..., 0]
    return {"o": o.reshape(B, Hq, nq, D).half(), "lse": lse.reshape(B, Hq, nq)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("extend", "release"):
        lens, other = _cases_lens(case)
        page = case["page"]
        if op == "extend":
            pages = sum(_pages(a + b, page) - _pages(a, page) for a, b in zip(lens, other))
            return {"bytes": 16 * case["B"] + 8 * pages + 8 * sum(other), "flops": 0}
        pages = sum(_pages(a, page) - _pages(b, page) for a, b in zip(lens, other))
        return {"bytes": 8 * case["B"] + 8 * pages, "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        rows = case["B"] * case["S"]
        return {"bytes": rows * ((Hq + Hkv) * D * 4 + 4 * case["axes"]),
                "flops": rows * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    if op == "append":
        rows = sum(_spread(case["B"], case["lo"], case["hi"]))
        elem = 1 if case["e4m3"] else 2
        return {"bytes": rows * (Hq * D * 4 + 2 * Hkv * D * (2 + elem) + 8),
                "flops": rows * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))}
    groups = _groups(case)
    members = sum(m for m, _ in groups)
    mine = _spread(members, case["lo"], case["hi"])
    tokens = sum(p for _, p in groups) + sum(mine)
    rows = members * Hq * case["nq"]
    pairs = Hq * case["nq"] * (sum(m * p for m, p in groups) + sum(mine))
    return {"bytes": 4 * D * Hkv * tokens + rows * (4 * D + 4), "flops": 4 * D * pairs}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"extend": _exact_extend, "release": _exact_release, "rope": _exact_rope,
                "append": _exact_append, "shared": _exact_shared}[s["op"]](s)


def _i64(values):
    return torch.tensor(np.asarray(values, dtype=np.int64), device="cuda")


def _exact_extend(s):
    table = s["page_table"].cpu().numpy().astype(np.int64)
    old, new = s["kv_lens"].tolist(), s["new_lens"].tolist()
    stack = s["free_pages"].tolist()[:int(s["free_count"])]
    page, lens, positions, slots, starts = s["page"], [], [], [], [0]
    full = False                     # the stack has run out: who needs a page gets nothing
    for b, (n, m) in enumerate(zip(old, new)):
        have = _pages(n, page)
        need = _pages(n + m, page) - have
        full = full or need > len(stack)
        t = np.arange(n, n + m)
        starts.append(starts[-1] + m)
        if full and need:
            lens.append(n)
            positions.append(np.full(m, -1))
            slots.append(np.full(m, -1))
            continue
        for p in range(have, have + need):
            table[b, p] = stack.pop()
        lens.append(n + m)
        positions.append(t)
        slots.append(table[b, t // page] * page + t % page)
    return {"page_table": _i64(table), "kv_lens": _i64(lens), "free_count": _i64([len(stack)]),
            "token_starts": _i64(starts), "positions": _i64(np.concatenate(positions)),
            "slots": _i64(np.concatenate(slots))}


def _exact_release(s):
    free, at = s["free_pages"].cpu().numpy().astype(np.int64), int(s["free_count"])
    table, page = s["page_table"].cpu().numpy(), s["page"]
    for b, (n, keep) in enumerate(zip(s["kv_lens"].tolist(), s["keep_lens"].tolist())):
        gone = table[b, _pages(keep, page):_pages(n, page)]
        free[at:at + len(gone)] = gone
        at += len(gone)
    return {"free_pages": _i64(free), "free_count": _i64([at])}


def _exact_turn(s, x, weight, axis_positions):
    """One head's rows x [S][D] in float64: the norm, then each pair as a complex number."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / torch.sqrt(torch.sum(x * x, -1, keepdim=True) / x.shape[-1] + EPS)
    rot = s["rot"]
    half = torch.arange(rot // 2, device="cuda")
    re, im = (2 * half, 2 * half + 1) if s["interleaved"] else (half, half + rot // 2)
    turn = torch.polar(torch.full_like(axis_positions, s["rope_scale"]),
                       axis_positions * s["freqs"].double())
    z = torch.complex(x[:, re], x[:, im]) * turn
    out = x.clone()
    out[:, re], out[:, im] = z.real, z.imag
    return out


def _exact_heads(s, x, weight):
    B, H, S, D = x.shape
    out = torch.empty((B, H, S, D), dtype=torch.float64, device="cuda")
    pos = s["positions"].reshape(-1, B, S)
    sizes = s.get("sections") or [s["rot"] // 2]
    for b in range(B):
        where = torch.cat([pos[i, b].double()[:, None].expand(S, n) for i, n in enumerate(sizes)], 1)
        for h in range(H):
            out[b, h] = _exact_turn(s, x[b, h], weight, where)
    return out


def _exact_rope(s):
    return {"q": _exact_heads(s, s["q"], s["q_weight"]), "k": _exact_heads(s, s["k"], s["k_weight"])}


def _exact_append(s):
    out = {"q": _exact_heads(s, s["q"], s["q_weight"])}
    page = s["page"]
    at = s["slots"][0].long()
    for name, x, scale in (("k_pages", _exact_heads(s, s["k"], s["k_weight"]), s["k_scale"]),
                           ("v_pages", s["v"].double(), s["v_scale"])):
        pages = _values(s, name).to(torch.float64)
        pages[at // page, at % page] = (x[0] / scale).clamp(-448, 448).permute(1, 0, 2) \
            if s["e4m3"] else x[0].permute(1, 0, 2)
        out[name] = pages
    return out


def _exact_shared(s):
    B, Hq, nq, D = s["q"].shape
    page, grp = s["page"], Hq // s["Hkv"]
    o = torch.zeros((B, Hq, nq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = s["prefix_of"][b] + s["own_lens"][b]
        if n == 0:
            continue
        used = s["page_table"][b, :_pages(n, page)].long()
        k = s["k_pages"][used].flatten(0, 1)[:n].double()
        v = s["v_pages"][used].flatten(0, 1)[:n].double()
        for h in range(Hq):
            for i in range(max(0, nq - n), nq):
                m = n - nq + i + 1
                x = k[:m, h // grp] @ s["q"][b, h, i].double() / math.sqrt(D)
                lse[b, h, i] = torch.logsumexp(x, 0)
                o[b, h, i] = torch.exp(x - lse[b, h, i]) @ v[:m, h // grp]
    return {"o": o, "lse": lse}
