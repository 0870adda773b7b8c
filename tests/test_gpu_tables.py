"""Page tables on the GPU (kv_paged_extend, kv_paged_release) against a stack popped and pushed page by
page; every result is exact."""

import numpy as np
import pytest
import torch

from oracle import tables as OT

pytestmark = pytest.mark.gpu
DEV = "cuda"


def t(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(lens, page, spare, width, seed, capacity=None, free=None):
    """(table, stack as a list, free_pages, count): every sequence holds its pages, -1 past them;
    `free` of the others are on the stack, `spare` pages beyond what the sequences hold exist."""
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in lens]
    P = sum(held) + spare
    order = rng.permutation(P).astype(np.int32)
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, c in enumerate(held):
        table[b, :c] = order[at:at + c]
        at += c
    stack = [int(p) for p in order[at:]][:free]
    pages = np.full(P if capacity is None else capacity, -7, dtype=np.int32)
    pages[:len(stack)] = stack
    return table, stack, pages, P


def run_extend(gb, lens, new, page, width, spare, seed=1, in_place=False, rows=None, pad=0, free=None,
               flags=0):
    table, stack, pages, P = make(lens, page, spare, width, seed, free=free)
    rt, rl, rs, tokens, refused = OT.extend(table, lens, new, stack, page)
    gt, gl, gp, gc = t(table), t(lens), t(pages), t([len(stack)])
    kw = dict(row_tokens=rows) if rows else dict(max_tokens=max(1, sum(new) + pad))
    if in_place:
        kw.update(kv_lens_out=gl, free_count_out=gc)
    old = gl.clone()
    out = gb.kv_paged_extend(gt, gl, t(new), gp, gc, page, P, **kw)
    assert gb.device_status() == (gb.DEV_NO_PAGES if refused else 0) | flags
    assert np.array_equal(gt.cpu().numpy(), rt)
    assert out[0].tolist() == rl and out[1].tolist() == [len(rs)]
    assert np.array_equal(gp.cpu().numpy(), pages)
    if in_place:
        assert out[0] is gl and out[1] is gc
    else:
        assert torch.equal(gl, old) and gc.tolist() == [len(stack)]
    if rows:
        pos, slots = OT.rows(tokens, rows)
    else:
        pos, slots, _ = OT.packed(tokens, kw["max_tokens"])
    assert out[2].tolist() == np.cumsum([0] + list(new)).tolist()
    assert np.array_equal(out[3].cpu().numpy(), pos) and np.array_equal(out[4].cpu().numpy(), slots)
    return refused


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_extend_ragged(gb, page, in_place):
    run_extend(gb, [0, 1, 15, 16, 17, 300, 0, 255], [1, 0, 1, 1, 40, 16, 700, 1], page, 64, 70,
               in_place=in_place)
    run_extend(gb, [0], [1], page, 1, 1, in_place=in_place)
    run_extend(gb, [33, 64, 0], [0, 0, 0], page, 8, 3, in_place=in_place, pad=5)


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_many_sequences_and_tokens(gb, in_place):
    rng = np.random.default_rng(5)
    for B, top in ((4096, 9), (1000, 130), (513, 2), (3, 40000)):
        lens = [int(x) for x in rng.integers(0, 500, B)]
        new = [int(x) for x in rng.integers(0, top + 1, B)]
        width = -(-(max(lens) + top) // 16) + 1
        run_extend(gb, lens, new, 16, width, sum(new) // 16 + B + 5, seed=B, in_place=in_place, pad=77)


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_rows(gb, in_place):
    run_extend(gb, [5, 0, 31, 32, 100], [3, 4, 0, 1, 2], 16, 9, 9, rows=4, in_place=in_place)
    run_extend(gb, [7] * 70, [1] * 70, 32, 3, 80, rows=1, in_place=in_place)
    run_extend(gb, [0, 10, 2000], [5000, 1234, 0], 64, 200, 150, rows=5000, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("free", [0, 1, 4, 5, 8])
def test_extend_with_too_few_pages(gb, free, in_place):
    """Sequences behind the one that does not fit get none either, unless they need none."""
    refused = run_extend(gb, [16, 3, 0, 30, 16, 8], [16, 2, 60, 3, 1, 8], 16, 8, 20, free=free,
                         in_place=in_place)
    assert bool(refused) == (free < 7)
    run_extend(gb, [16, 3, 0, 30, 16, 8], [16, 2, 60, 3, 1, 8], 16, 8, 20, free=free, rows=60,
               in_place=in_place)


def test_extend_without_maps(gb):
    table, stack, pages, P = make([40, 0], 16, 12, 10, 3)
    gt, gl = t(table), t([40, 0])
    lens, count, starts, pos, slots = gb.kv_paged_extend(gt, gl, t([30, 99]), t(pages),
                                                         t([len(stack)]), 16, P)
    rt, rl, rs, _, _ = OT.extend(table, [40, 0], [30, 99], stack, 16)
    assert np.array_equal(gt.cpu().numpy(), rt) and lens.tolist() == rl and count.item() == len(rs)
    assert starts is None and pos is None and slots is None and gb.device_status() == 0


def test_extend_fewer_entries_than_tokens(gb):
    """The first max_tokens are written, and nothing behind the arrays."""
    table, stack, pages, P = make([10, 20, 30], 16, 40, 20, 4)
    new = [100, 50, 60]
    store = torch.full((2, 140), 77, dtype=torch.int32, device=DEV)
    gt = t(table)
    gb.kv_paged_extend(gt, t([10, 20, 30]), t(new), t(pages), t([len(stack)]), 16, P, max_tokens=120,
                       positions=store[0, :120], slots=store[1, :120])
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    rt, _, _, tokens, _ = OT.extend(table, [10, 20, 30], new, stack, 16)
    pos, slots, _ = OT.packed(tokens, 120)
    got = store.cpu().numpy()
    assert np.array_equal(got[:, :120], [pos, slots]) and (got[:, 120:] == 77).all()
    assert np.array_equal(gt.cpu().numpy(), rt)


@pytest.mark.parametrize("in_place", [False, True])
def test_extend_bad_lengths(gb, in_place):
    """Lengths out of range leave their sequences as they are and take no places."""
    lens = [16, -1, 161, 30, 100, 10, 2 ** 31 - 1, 20]
    new = [1, 5, 1, -3, 61, 5, 2 ** 31 - 1, 2 ** 31 - 1]
    good = [0, 5]
    table, stack, pages, P = make([16, 0, 0, 30, 100, 10, 0, 20], 16, 9, 10, 6)
    gt, gl, gc = t(table), t(lens), t([len(stack)])
    kw = dict(kv_lens_out=gl, free_count_out=gc) if in_place else {}
    out = gb.kv_paged_extend(gt, gl, t(new), t(pages), gc, 16, P, max_tokens=9, **kw)
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    rt, rl, rs, tokens, _ = OT.extend(table[good], [16, 10], [1, 5], stack, 16)
    want = list(lens)
    want[0], want[5] = rl
    assert out[0].tolist() == want and out[1].item() == len(rs)
    full = table.copy()
    full[good] = rt
    assert np.array_equal(gt.cpu().numpy(), full)
    pos, slots, _ = OT.packed(tokens, 9)
    assert out[3].tolist() == pos.tolist() and out[4].tolist() == slots.tolist()
    assert out[2].tolist() == [0, 1, 1, 1, 1, 1, 6, 6, 6]
    # a count that is none
    for bad in (-1, P + 1):
        out = gb.kv_paged_extend(t(table), t([16] * 8), t([1] * 8), t(pages), t([bad]), 16, P)
        assert gb.device_status() == gb.DEV_BAD_LENGTH | gb.DEV_NO_PAGES
        assert out[0].tolist() == [16] * 8 and out[1].item() == 0


def test_extend_bad_pages(gb):
    """A page that is none, in the row or on the stack: its tokens have no slot."""
    pages = [5, 99, -1, 3]
    table = t([[7, -1, -1], [8, -1, -1], [-1, -1, -1]])
    out = gb.kv_paged_extend(table, t([16, 16, 2]), t([2, 2, 2]), t(pages), t([4]), 16, 9,
                             max_tokens=6)
    assert gb.device_status() == gb.DEV_BAD_PAGE
    assert out[4].tolist() == [48, 49, -1, -1, -1, -1]
    assert out[3].tolist() == [16, 17, 16, 17, 2, 3] and out[0].tolist() == [18, 18, 4]


def run_release(gb, lens, keep, page, width, seed=1, in_place=False, free=3, capacity=None):
    table, stack, pages, P = make(lens, page, free + 4, width, seed, capacity=capacity, free=free)
    given_keep = [0] * len(lens) if keep is None else keep
    rs = OT.release(table, lens, given_keep, stack, page, len(pages))
    gp, gc = t(pages), t([len(stack)])
    kw = dict(free_count_out=gc) if in_place else {}
    out = gb.kv_paged_release(t(table), t(lens), gp, gc, page, P,
                              keep_lens=None if keep is None else t(keep), **kw)
    total = len(stack) + sum(-(-n // page) + (-k // page) for n, k in zip(lens, given_keep))
    assert gb.device_status() == (gb.DEV_NO_PAGES if total > len(pages) else 0)
    want = pages.copy()
    want[:len(rs)] = rs
    assert out.item() == len(rs) and np.array_equal(gp.cpu().numpy(), want)
    if not in_place:
        assert gc.item() == len(stack)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_release(gb, page, in_place):
    lens = [0, 1, 16, 17, 300, 255, 256, 700]
    run_release(gb, lens, None, page, 60, in_place=in_place)
    run_release(gb, lens, [0, 1, 0, 16, 17, 255, 1, 130], page, 60, in_place=in_place)
    run_release(gb, lens, lens, page, 60, in_place=in_place)
    run_release(gb, [5], [0], page, 1, in_place=in_place, free=0)


@pytest.mark.parametrize("in_place", [False, True])
def test_release_many(gb, in_place):
    rng = np.random.default_rng(8)
    for B, top in ((4096, 60), (70, 20000), (2, 1300000)):
        lens = [int(x) for x in rng.integers(0, top, B)]
        keep = [int(rng.integers(0, n + 1)) for n in lens]
        run_release(gb, lens, keep, 16, top // 16 + 1, seed=B, in_place=in_place)
        run_release(gb, lens, None, 16, top // 16 + 1, seed=B, in_place=in_place)


@pytest.mark.parametrize("capacity", [3, 4, 9, 10, 12, 13])
def test_release_onto_a_full_stack(gb, capacity):
    """Pages of a sequence go all or none; behind one that does not fit, none."""
    run_release(gb, [16, 0, 90, 30, 16], None, 16, 8, capacity=capacity)


def test_release_bad_lengths_and_pages(gb):
    lens = [40, -1, 40, 200, 40, 40]
    keep = [0, 0, 41, 0, -1, 17]
    table = np.arange(36, dtype=np.int32).reshape(6, 6)
    pages = t([77] * 60)
    out = gb.kv_paged_release(t(table), t(lens), pages, t([2]), 16, 100, keep_lens=t(keep))
    assert gb.device_status() == gb.DEV_BAD_LENGTH
    assert out.item() == 6 and pages.tolist()[:7] == [77, 77, 0, 1, 2, 32, 77]
    # a sequence with a bad page keeps all of its pages, the others' move up
    for many in (6, 3000):
        B = many
        table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
        table[1, 2], table[B - 2, 0], table[3, 3] = -1, 4 * B, -5     # [3, 3] is not given back
        pages = t([77] * (4 * B + 9))
        out = gb.kv_paged_release(t(table), t([48] * B), pages, t([5]), 16, 4 * B)
        assert gb.device_status() == gb.DEV_BAD_PAGE
        want = [p for b in range(B) if b not in (1, B - 2) for p in table[b, :3].tolist()]
        got = pages.tolist()
        assert out.item() == 5 + len(want) and got[5:5 + len(want)] == want
        assert set(got[:5]) == {77} and set(got[5 + len(want):]) == {77}
    for bad in (-1, 61):
        pages = t([77] * 60)
        out = gb.kv_paged_release(t(table[:1]), t([48]), pages, t([bad]), 16, 4 * many)
        assert gb.device_status() == gb.DEV_BAD_LENGTH
        assert out.item() == 3 and pages.tolist()[:4] == [0, 1, 2, 77]


def test_steps_in_a_graph_carry_their_state(gb):
    """Two captured steps on a side stream: tokens come and half of them go, replayed."""
    lens, page, width = [0, 20, 31], 16, 40
    table, stack, pages, P = make(lens, page, 60, width, 9)
    gt, gl, gp, gc = t(table), t(lens), t(pages), t([len(stack)])
    new, keep = t([9, 33, 1]), torch.empty(3, dtype=torch.int32, device=DEV)
    pos = torch.empty((3, 33), dtype=torch.int32, device=DEV)
    slots, starts = torch.empty_like(pos), torch.empty(4, dtype=torch.int32, device=DEV)

    def step():
        gb.kv_paged_extend(gt, gl, new, gp, gc, page, P, row_tokens=33, kv_lens_out=gl,
                           free_count_out=gc, positions=pos, slots=slots, token_starts=starts)
        torch.sub(gl, new // 2, out=keep)
        gb.kv_paged_release(gt, gl, gp, gc, page, P, keep_lens=keep, free_count_out=gc)
        gl.copy_(keep)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(7):
        graph.replay()
        table, lens, stack, tokens, refused = OT.extend(table, lens, [9, 33, 1], stack, page)
        kept = [n - m // 2 for n, m in zip(lens, [9, 33, 1])]
        stack = OT.release(table, lens, kept, stack, page, len(pages))
        lens = kept
        torch.cuda.synchronize()
        rp, rs = OT.rows(tokens, 33)
        assert not refused and gl.tolist() == lens and gc.item() == len(stack)
        assert np.array_equal(pos.cpu().numpy(), rp) and np.array_equal(slots.cpu().numpy(), rs)
        assert gp.tolist()[:len(stack)] == stack and np.array_equal(gt.cpu().numpy(), table)
    assert gb.device_status() == 0
