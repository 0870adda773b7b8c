"""Page tables, rotary positions and decode behind shared prefixes at their edges: guard bands around every output,
splits of every size, calls at the same time on two streams, strided views, arguments that are the
same tensor."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs
from oracle import paged as OP
from oracle import rope as OR
from oracle import tables as OT
from test_gpu_guards import Guarded
from test_gpu_guards_f16 import guarded
from tests.test_gpu_decode_shared import check, shared_inputs, widen
from tests.test_gpu_paged_f16 import assert_within, row_error
from tests.test_gpu_rope import close, inputs_of, t
from tests.test_gpu_tables import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- decode behind shared prefixes

def workspaces(gb, x):
    """Bytes of the full-speed workspace, and those below which the call is refused (which the host decides)."""
    q, kp, vp, call, _, lens, starts, pre = x
    a = [t(y) for y in (q, kp, vp, widen(call), lens, starts, pre)]
    most = a[3].shape[1] * kp.shape[1]
    lo, hi = 0, gb.attn_paged_decode_shared_f16_workspace_size(*q.shape[:2], kp.shape[2], q.shape[2], len(pre), most,
                                                               most, q.shape[3])
    full, ws = hi, torch.empty(hi, dtype=torch.uint8, device=DEV)
    while hi - lo > 16:
        mid = (lo + hi) // 2
        try:
            gb.attn_paged_decode_shared_f16_fwd(*a, workspace=ws[:mid])
            hi = mid
        except gb.GbattnError as e:
            assert e.status == 6
            lo = mid
    return full, hi


def over_splits(gb, x, parts):
    """The form of two kernels with workspaces from the smallest (two CTAs) to the full one, each in guard bands."""
    q, kp, vp, call, whole, lens, starts, pre = x
    full, least = workspaces(gb, x)
    ref = OP.decode(q, kp, vp, whole, lens, inputs.softmax_scale(q.shape[3]))
    e = row_error(ref["size"], q.shape[3])
    a = [t(y) for y in (q, kp, vp, widen(call), lens, starts, pre)]
    for part in parts:
        ws = Guarded((int(least + part * (full - least)) // 4 + 1,), torch.int32)
        lse = torch.full(q.shape[:3], 7.0, device=DEV)
        o = gb.attn_paged_decode_shared_f16_fwd(*a, lse=lse, workspace=ws.view)
        assert gb.device_status() == 0 and ws.intact()
        assert_within(o.float().cpu().numpy(), ref["o"],
                      2.0 ** -11 * np.abs(ref["o"]) + 2.0 ** -25 + 2 * e[..., None] * ref["spread"], f"o, {part}")
        with np.errstate(invalid="ignore"):
            assert_within(lse.cpu().numpy(), ref["lse"], e + 2.0 ** -23 * np.abs(ref["lse"]), f"lse, {part}")


@pytest.mark.parametrize("D,Hq", [(128, 8), (64, 8), (256, 8)])
def test_groups_of_unlike_units(gb, D, Hq):
    """A group whose last unit is shorter than its others, beside groups of one unit: the split into ranges must
    be the same in the decode and in the merge."""
    for groups in ([(40, 2048), (16, 2048)], [(16, 1024), (33, 4096), (2, 0)]):
        B = sum(m for m, _ in groups)
        x = shared_inputs(groups, [(5 * i) % 40 for i in range(B)], Hq, 1, 1, D, 64, 31)
        over_splits(gb, x, [0.0] + [i / 40 for i in range(1, 12)])


@pytest.mark.parametrize("seed", range(12))
def test_splits_of_every_size(gb, seed):
    """Random groups over random numbers of CTAs."""
    rng = np.random.default_rng(200 + seed)
    D = (64, 128, 256)[seed % 3]
    Hkv = int(rng.integers(1, 4))
    Hq, nq = Hkv * int(rng.integers(1, 13)), int(rng.integers(1, 3))
    groups = [(int(rng.integers(0, 30)), 16 * int(rng.integers(0, 120))) for _ in range(int(rng.integers(1, 6)))]
    groups.append((1, 64))
    own = [int(rng.integers(0, 200)) for _ in range(sum(m for m, _ in groups))]
    x = shared_inputs(groups, own, Hq, Hkv, nq, D, 16, seed)
    over_splits(gb, x, [0.0, *rng.random(6).tolist(), 1.0])


def test_workspace_and_outputs_in_guard_bands(gb):
    for D, Hq, Hkv, nq in ((64, 3, 1, 1), (128, 12, 2, 2), (256, 5, 1, 3)):
        x = shared_inputs([(3, 336), (1, 0), (20, 48)], [5, 0, 333] + [17] * 21, Hq, Hkv, nq, D, 16, D, poison=False)
        q, kp, vp, call, _, lens, starts, pre = x
        want = None
        for table in (call, widen(call)):
            most = table.shape[1] * 16
            kw = {} if table is not call else dict(max_prefix_len=336, max_own_len=333)
            size = gb.attn_paged_decode_shared_f16_workspace_size(
                24, Hq, Hkv, nq, 3, kw.get("max_prefix_len", most), kw.get("max_own_len", most), D)
            o, lse, ws = Guarded(q.shape, torch.float16), Guarded(q.shape[:3], torch.float32), \
                Guarded((-(-size // 4),), torch.int32)
            k, v = guarded(kp), guarded(vp)
            gb.attn_paged_decode_shared_f16_fwd(t(q), k.view, v.view, t(table), t(lens), t(starts), t(pre), o=o.view,
                                                lse=lse.view, workspace=ws.view, **kw)
            assert gb.device_status() == 0 and all(g.intact() for g in (o, lse, ws, k, v))
            assert np.array_equal(k.view.cpu().numpy(), kp) and np.array_equal(v.view.cpu().numpy(), vp)
            got = o.view.float().clone()
            assert want is None or (got - want).abs().max() <= 2.0 ** -9 * want.abs().max()
            want = got


def test_many_query_rows(gb):
    """Drafts of hundreds of tokens: more rows of one sequence than a unit holds."""
    check(gb, [(2, 512), (1, 0)], [400, 3, 350], 2, 1, 350, 128, 16, seed=41)
    check(gb, [(2, 512), (1, 64)], [400, 3, 350], 8, 2, 130, 256, 32, seed=42)


def test_two_streams_at_once(gb):
    """Separate workspaces, one stream each: bit for bit what each call gives alone."""
    xs = [shared_inputs([(12, 4096), (3, 512)], [(61 * i) % 700 for i in range(15)], 16, 2, 1, 128, 64, 51),
          shared_inputs([(1, 1024), (30, 2048)], [(37 * i) % 900 for i in range(31)], 8, 1, 2, 64, 16, 52)]
    args = [[t(y) for y in (x[0], x[1], x[2], x[3], x[5], x[6], x[7])] for x in xs]
    def sizes(a):
        most = a[3].shape[1] * a[1].shape[1]
        return (a[0].shape[0], a[0].shape[1], a[1].shape[2], a[0].shape[2], a[6].shape[0], most, most, a[0].shape[3])
    ws = [torch.empty(gb.attn_paged_decode_shared_f16_workspace_size(*sizes(a)), dtype=torch.uint8, device=DEV)
          for a in args]
    alone = [gb.attn_paged_decode_shared_f16_fwd(*a, workspace=w).clone() for a, w in zip(args, ws)]
    outs = [[torch.empty_like(o) for _ in range(20)] for o in alone]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for i in range(20):
        for a, w, o, s in zip(args, ws, outs, streams):
            gb.attn_paged_decode_shared_f16_fwd(*a, o=o[i], workspace=w, stream=s)
    torch.cuda.synchronize()
    assert gb.device_status() == 0
    for want, got in zip(alone, outs):
        assert all(torch.equal(want, g) for g in got)


# ---------------------------------------------------------------- page tables

def test_table_outputs_in_guard_bands(gb):
    lens, new, page = [0, 40, 31, 64, 5], [33, 0, 1, 16, 300], 16
    table, stack, pages, P = make(lens, page, 60, 24, 1)
    rt, rl, rs, tokens, _ = OT.extend(table, lens, new, stack, page)
    pos, slots, _ = OT.packed(tokens, 360)
    for in_place in (False, True):
        gt, gp = guarded(table), guarded(pages)
        gl, gc = guarded(np.array(lens, np.int32)), guarded(np.array([len(stack)], np.int32))
        out = [gl, gc] if in_place else [Guarded((5,), torch.int32), Guarded((1,), torch.int32)]
        out += [Guarded((6,), torch.int32), Guarded((360,), torch.int32), Guarded((360,), torch.int32)]
        gb.kv_paged_extend(gt.view, gl.view, t(np.array(new, np.int32)), gp.view, gc.view, page, P, max_tokens=360,
                           kv_lens_out=out[0].view, free_count_out=out[1].view, token_starts=out[2].view,
                           positions=out[3].view, slots=out[4].view)
        assert gb.device_status() == 0 and all(g.intact() for g in (gt, gp, gl, gc, *out))
        assert np.array_equal(gt.view.cpu().numpy(), rt) and out[0].view.tolist() == rl
        assert out[1].view.tolist() == [len(rs)] and np.array_equal(gp.view.cpu().numpy(), pages)
        assert np.array_equal(out[3].view.cpu().numpy(), pos) and np.array_equal(out[4].view.cpu().numpy(), slots)
        # and all of it back, onto a stack with exactly that much room
        back = guarded(np.array(list(rs) + [-7] * (len(stack) - len(rs)), np.int32))
        count = guarded(np.array([len(rs)], np.int32))
        gb.kv_paged_release(gt.view, out[0].view, back.view, count.view, page, P, keep_lens=t(np.array(lens, np.int32)),
                            free_count_out=count.view)
        assert gb.device_status() == 0 and back.intact() and count.intact() and gt.intact()
        assert count.view.tolist() == [len(stack)] and sorted(back.view.tolist()) == sorted(stack)
        assert np.array_equal(gt.view.cpu().numpy(), rt)


@pytest.mark.parametrize("lens_in_place", [False, True])
def test_one_of_the_two_in_place(gb, lens_in_place):
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 300, 900)]
    new = [int(n) for n in rng.integers(0, 60, 900)]
    table, stack, pages, P = make(lens, 32, 3000, 16, 4)
    rt, rl, rs, tokens, _ = OT.extend(table, lens, new, stack, 32)
    pos, slots, _ = OT.packed(tokens, sum(new))
    gt, gl, gc = (t(np.asarray(x, dtype=np.int32)) for x in (table, lens, [len(stack)]))
    kw = dict(kv_lens_out=gl) if lens_in_place else dict(free_count_out=gc)
    out = gb.kv_paged_extend(gt, gl, t(np.array(new, np.int32)), t(pages), gc, 32, P, max_tokens=sum(new), **kw)
    assert gb.device_status() == 0 and np.array_equal(gt.cpu().numpy(), rt)
    assert out[0].tolist() == rl and out[1].tolist() == [len(rs)]
    assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)
    assert gl.tolist() == (rl if lens_in_place else lens) and gc.tolist() == [len(stack) if lens_in_place else len(rs)]


def test_lengths_as_two_arguments(gb):
    """Every sequence doubled (new_lens is kv_lens), and none shortened (keep_lens is kv_lens)."""
    lens = [16, 0, 7, 100]
    table, stack, pages, P = make(lens, 16, 20, 16, 6)
    rt, rl, rs, _, _ = OT.extend(table, lens, lens, stack, 16)
    gt, gl, gp, gc = (t(np.asarray(x, dtype=np.int32)) for x in (table, lens, pages, [len(stack)]))
    out = gb.kv_paged_extend(gt, gl, gl, gp, gc, 16, P)
    assert np.array_equal(gt.cpu().numpy(), rt) and out[0].tolist() == rl and out[1].tolist() == [len(rs)]
    assert gb.kv_paged_release(gt, out[0], gp, gc, 16, P, keep_lens=out[0]).tolist() == [len(stack)]
    assert np.array_equal(gp.cpu().numpy(), pages) and gb.device_status() == 0
    with pytest.raises(gb.GbattnError):   # written while others read it
        gb.kv_paged_extend(gt, gl, gl, gp, gc, 16, P, kv_lens_out=gl)


@pytest.mark.parametrize("B,width", [(300, 600), (33, 8000)])
def test_bad_pages_among_very_many(gb, B, width):
    """More pages than the cluster keeps in registers at once: sequences with a bad one, first or last looked at, keep
    all of theirs."""
    rng = np.random.default_rng(B)
    P = B * width
    table = rng.permutation(P).astype(np.int32).reshape(B, width)
    lens = rng.integers(0, 16 * width + 1, B)
    lens[[0, 5, B - 1]] = 16 * width
    bad = sorted({0, 5, B - 1, *rng.integers(0, B, 4).tolist()})
    for b in bad:
        held = -(-int(lens[b]) // 16)
        if held:
            table[b, rng.choice([0, held - 1, held // 2])] = rng.choice([-1, P, 2 ** 31 - 1])
    count, pages = t(np.array([3], np.int32)), t(np.full(P + 5, 77, np.int32))
    out = gb.kv_paged_release(t(table), t(lens.astype(np.int32)), pages, count, 16, P)
    assert gb.device_status() == gb.DEV_BAD_PAGE
    want = np.concatenate([table[b, :-(-int(lens[b]) // 16)] for b in range(B) if b not in bad])
    got = pages.cpu().numpy()
    assert out.item() == 3 + len(want) and np.array_equal(got[3:3 + len(want)], want)
    assert (got[:3] == 77).all() and (got[3 + len(want):] == 77).all()


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("D,rot,inter", [(64, 24, False), (128, 128, True), (256, 72, False)])
def test_strided_rows_and_what_lies_between(gb, D, rot, inter):
    """Inputs and outputs with gaps between rows, heads and batch entries: the gaps stay as they are."""
    q, k, _, pos, freqs, w, _ = inputs_of(3, 3, 2, 13, D, rot, 1, True, 4000, D)
    def wide(x, fill):
        B, H, S, _ = x.shape
        buf = torch.full((B, S + 2, H + 3, D + 24), fill, dtype=torch.float16, device=DEV)
        view = buf[:, 1:S + 1, 2:H + 2, 8:D + 8].permute(0, 2, 1, 3)
        return buf, view
    ins = [wide(x, float("nan")) for x in (q, k)]
    outs = [wide(x, -7776.0) for x in (q, k)]
    for (_, view), x in zip(ins, (q, k)):
        view.copy_(t(x))
    gb.qk_norm_rope_f16(ins[0][1], ins[1][1], t(pos[0]), t(freqs), q_weight=t(w[0]), k_weight=t(w[1]),
                        interleaved=inter, q_out=outs[0][1], k_out=outs[1][1])
    assert gb.device_status() == 0
    for (buf, view), x, weight in zip(outs, (q, k), w):
        ref, size = OR.rotate(x, pos, freqs, weight, interleaved=inter)
        close(view.cpu().numpy(), ref, size, "rows")
        view.fill_(-7776.0)
        assert (buf == -7776.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_pools_in_guard_bands(gb, e4m3):
    q, k, v, pos, freqs, w, _ = inputs_of(1, 3, 1, 33, 64, 64, 1, True, 100, 7)
    P, page = 3, 16
    slots = np.arange(P * page, dtype=np.int32)[::-1][:33].reshape(1, 33)   # the pool's last slot among them
    dtype = torch.uint8 if e4m3 else torch.float16
    fill = 129 if e4m3 else -7776.0
    bufs = [torch.full((4096 + P * page * 64 + 4096,), fill, dtype=dtype, device=DEV) for _ in range(2)]
    pools = [b[4096:-4096].view(P, page, 1, 64) for b in bufs]
    gw, out = Guarded((P, 1, page), torch.float32), Guarded((1, 3, 33, 64), torch.float16)
    gb.kv_paged_rope_append(t(q), t(k), t(v), t(slots), *pools, t(pos[0]), t(freqs), q_weight=t(w[0]),
                            weights=gw.view, q_out=out.view)
    assert gb.device_status() == 0 and gw.intact() and out.intact()
    for b, p in zip(bufs, pools):
        assert (b[:4096] == fill).all() and (b[-4096:] == fill).all()
        rows = p.view(-1, 64)
        assert (rows[:P * page - 33] == fill).all() and not (rows[P * page - 33:] == fill).all(1).any()
    flat = gw.view.view(-1)
    assert (flat[:P * page - 33] == -7776).all() and (flat[P * page - 33:] == 0).all()
    ref, size = OR.rotate(q, pos, freqs, w[0])
    close(out.view.cpu().numpy(), ref, size, "q")
