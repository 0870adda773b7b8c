"""Refusals of the page-table and rotary calls (CPU only): arguments are checked before any CUDA call, so
placeholder addresses reach every branch; valid arguments end in GBATTN_ERR_CUDA where no GPU is
visible.  The oracles' pins and the frequencies of long contexts."""

import ctypes
import math

import numpy as np
import pytest

from oracle import rope as OR, tables as OT
from tests.test_abi_paged import (ALIAS, ALIGN, CUDA, MIS2, MIS8, NULL, OK, SCALE, SHAPE, UNSUPPORTED,
                                  WORKSPACE, A, caller, lib)

assert lib


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def at(i, elements):
    """An address that many FP16 elements behind A(i)."""
    return ctypes.c_void_p(A(i).value + 2 * elements)


EXTEND = ("table", "lens", "new", "free", "count", "lens_out", "count_out", "starts", "pos", "slots", "B",
          "mp", "ps", "P", "cap", "rows", "tokens", "stream")


def test_extend_refusals(lib):
    base = dict(zip(EXTEND, [A(i) for i in range(10)] + [4, 8, 16, 32, 32, 0, 20, None]))
    call = caller(lib.kv_paged_extend, EXTEND, base)
    for n in ("table", "lens", "new", "free", "count", "lens_out", "count_out"):
        assert call(**{n: None}) == NULL
    assert call(pos=None) == NULL and call(slots=None) == NULL
    for n in ("B", "mp", "ps", "P", "cap"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(rows=-1) == SHAPE and call(tokens=-1) == SHAPE and call(tokens=0) == SHAPE
    assert call(rows=4) == SHAPE and call(rows=5) in (OK, CUDA) and call(rows=2 ** 30) == SHAPE
    assert call(B=4097) == UNSUPPORTED and call(ps=24) == UNSUPPORTED and call(ps=8) == UNSUPPORTED
    assert call(P=1 << 27) == UNSUPPORTED and call(mp=(1 << 26) + 1) == SHAPE
    assert call(B=1024, mp=(1 << 20) + 1) == SHAPE
    for n in EXTEND[:10]:
        assert call(**{n: MIS2}) == ALIGN
    for n in ("lens_out", "count_out", "starts", "pos", "slots"):
        assert call(**{n: A(0)}) == ALIAS and call(**{n: A(2)}) == ALIAS and call(**{n: A(3)}) == ALIAS
    assert call(table=A(3)) == ALIAS and call(pos=A(9)) == ALIAS and call(lens_out=A(4)) == ALIAS
    assert call(count_out=A(1)) == ALIAS and call(lens_out=at(1, 2)) == ALIAS
    assert call(lens_out=A(1), count_out=A(4)) in (OK, CUDA) and call(starts=None) in (OK, CUDA)
    assert call(pos=None, slots=None, tokens=0) in (OK, CUDA) and call() in (OK, CUDA)


def test_release_refusals(lib):
    names = ("table", "lens", "keep", "free", "count", "count_out", "B", "mp", "ps", "P", "cap", "stream")
    base = dict(zip(names, [A(i) for i in range(6)] + [4, 8, 16, 32, 32, None]))
    call = caller(lib.kv_paged_release, names, base)
    for n in ("table", "lens", "free", "count", "count_out"):
        assert call(**{n: None}) == NULL
    for n in ("B", "mp", "ps", "P", "cap"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(B=4097) == UNSUPPORTED and call(ps=48) == UNSUPPORTED and call(P=1 << 27) == UNSUPPORTED
    for n in names[:6]:
        assert call(**{n: MIS2}) == ALIGN
    assert call(free=A(0)) == ALIAS and call(free=A(1)) == ALIAS and call(free=A(4)) == ALIAS
    assert call(count_out=A(2)) == ALIAS and call(count_out=A(3)) == ALIAS
    assert call(count_out=A(4)) in (OK, CUDA) and call(keep=None) in (OK, CUDA) and call() in (OK, CUDA)


ROPE = ("q", "k", "pos", "freqs", "qw", "kw", "qo", "ko", "B", "Hq", "Hk", "S", "D", "rot", "inter", "axes",
        "sections", "qs", "ks", "qos", "kos", "eps", "scale", "stream")


def sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


def test_rope_refusals(lib):
    base = dict(zip(ROPE, [A(i) for i in range(8)] + [2, 4, 2, 30, 128, 128, 0, 1, None, None, None, None,
                                                      None, 1e-6, 1.0, None]))
    call = caller(lib.qk_norm_rope_f16, ROPE, base)
    for n in ("q", "qo", "k", "ko", "pos", "freqs"):
        assert call(**{n: None}) == NULL
    assert call(k=None, ko=None) == NULL               # keys counted but not there
    for n in ("B", "Hq", "S", "Hk"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(rot=-8) == SHAPE and call(rot=136) == SHAPE and call(inter=2) == SHAPE
    assert call(axes=0) == SHAPE and call(axes=4) == SHAPE and call(axes=2) == NULL
    assert call(axes=2, sections=sections(30, 33)) == SHAPE
    assert call(axes=2, sections=sections(65, -1)) == SHAPE
    assert call(sections=sections(63)) == SHAPE and call(B=2 ** 30, S=4) == SHAPE
    for d in (0, 32, 96, 512):
        assert call(D=d) == UNSUPPORTED
    assert call(rot=20) == UNSUPPORTED
    for x in (0.0, -1.0, math.nan, math.inf):
        assert call(eps=x) == SCALE and call(scale=x) == SCALE
    for n in ("q", "k", "qo", "ko"):
        assert call(**{n: MIS8}) == ALIGN
    for n in ("pos", "freqs", "qw", "kw"):
        assert call(**{n: MIS2}) == ALIGN
    for n in ("qs", "ks", "qos", "kos"):
        assert call(**{n: strides(1, 2, 3)}) == SHAPE
    assert call(qos=strides(30 * 128, 0, 128)) == SHAPE
    assert call(qo=A(1)) == ALIAS and call(ko=A(0)) == ALIAS and call(qo=A(7)) == ALIAS
    assert call(qo=at(0, 8)) == ALIAS and call(qo=A(2)) == ALIAS and call(ko=A(3)) == ALIAS
    assert call(qo=A(4)) == ALIAS and call(qo=A(0), qos=strides(4 * 30 * 128, 128, 4 * 128)) == ALIAS
    good = (OK, CUDA)
    assert call(qo=A(0)) in good and call(qo=A(0), ko=A(1)) in good
    assert call(k=None, ko=None, Hk=0) in good and call(axes=3, sections=sections(32, 16, 16)) in good
    assert call(rot=0, pos=None, freqs=None, scale=0.0) in good
    assert call(rot=0, axes=3, freqs=None) in good and call(rot=0, sections=sections(9)) in good
    assert call(qw=None, kw=None, eps=0.0) in good and call(axes=2, sections=sections(0, 64)) in good
    # heads of one packed tensor [B][S][4 + 2 + 2][128]: apart, and not
    row = 8 * 128
    st = strides(30 * row, 128, row)
    inside = dict(qs=st, ks=st, qos=st, kos=st)
    assert call(k=at(0, 4 * 128), qo=A(0), ko=at(0, 4 * 128), **inside) in good
    assert call(k=at(0, 3 * 128), qo=A(0), ko=at(0, 3 * 128), **inside) == ALIAS
    assert call(k=at(0, 7 * 128), qo=A(0), ko=at(0, 7 * 128), **inside) == ALIAS    # into the next row
    assert call(k=at(0, 6 * 128), qo=A(0), ko=at(0, 6 * 128), **inside) in good
    assert call(k=at(0, 4 * 128), q=A(2), qo=A(0), ko=A(7), pos=A(9), qs=st, ks=st, qos=st,
                kos=None) in good
    one = strides(row, 128, 64)                        # one token a sequence: rows by batch entry
    inside = dict(S=1, qs=one, ks=one, qos=one, kos=one)
    assert call(k=at(0, 4 * 128), qo=A(0), ko=at(0, 4 * 128), **inside) in good
    assert call(k=at(0, 2 * 128), qo=A(0), ko=at(0, 2 * 128), **inside) == ALIAS
    other = strides(30 * row + 8, 128, row)            # batch entries not whole rows apart
    inside = dict(qs=other, ks=other, qos=other, kos=other)
    assert call(k=at(0, 4 * 128), qo=A(0), ko=at(0, 4 * 128), **inside) == ALIAS


APPEND = ("q", "k", "v", "slots", "pos", "freqs", "qw", "kw", "qo", "kp", "vp", "w", "B", "Hq", "Hkv", "S",
          "D", "rot", "inter", "axes", "sections", "qs", "kvs", "qos", "elem", "P", "ps", "eps", "scale",
          "k_scale", "v_scale", "stream")


def test_rope_append_refusals(lib):
    base = dict(zip(APPEND, [A(i) for i in range(12)] + [2, 4, 2, 30, 128, 64, 0, 1, None, None, None, None,
                                                         1, 16, 16, 1e-6, 1.0, 0.5, 0.25, None]))
    call = caller(lib.kv_paged_rope_append, APPEND, base)
    for n in ("q", "k", "v", "slots", "pos", "freqs", "qo", "kp", "vp"):
        assert call(**{n: None}) == NULL
    for n in ("B", "Hq", "Hkv", "S", "P", "ps"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    for kw in (dict(elem=4), dict(ps=24), dict(ps=8), dict(P=1 << 27), dict(D=96), dict(rot=12)):
        assert call(**kw) == UNSUPPORTED
    for x in (0.0, math.nan, math.inf):
        assert call(k_scale=x) == SCALE and call(v_scale=x) == SCALE
    for n in ("q", "k", "v", "qo", "kp", "vp"):
        assert call(**{n: MIS8}) == ALIGN
    for n in ("slots", "pos", "freqs", "qw", "kw", "w"):
        assert call(**{n: MIS2}) == ALIGN
    for n in ("qo", "kp", "vp", "w"):
        for i in (0, 1, 2, 3, 4, 5, 6):
            assert call(**{n: A(i)}) == (ALIAS if (n, i) != ("qo", 0) else call()), (n, i)
    assert call(vp=A(9)) == ALIAS and call(w=A(10)) == ALIAS and call(qo=A(9)) == ALIAS
    assert call() in (OK, CUDA) and call(elem=2, k_scale=0.0, v_scale=0.0, w=None) in (OK, CUDA)
    assert call(rot=0, pos=None, freqs=None) in (OK, CUDA)


SHARED = ("q", "kp", "vp", "table", "lens", "starts", "pre", "o", "lse", "B", "Hq", "Hkv", "nq", "D",
          "groups", "P", "ps", "mp", "maxp", "maxo", "scale", "ws", "wsb", "stream")


def test_shared_decode_refusals(lib):
    base = dict(zip(SHARED, [A(i) for i in range(9)] + [4, 4, 2, 1, 128, 2, 16, 16, 8, 64, 128, 0.1, A(20),
                                                        1 << 28, None]))
    call = caller(lib.attn_paged_decode_shared_f16_fwd, SHARED, base)
    for n in SHARED[:8]:
        assert call(**{n: None}) == NULL
    for n in ("B", "Hq", "Hkv", "nq", "groups", "P", "ps", "mp"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(maxp=-1) == SHAPE and call(maxo=-1) == SHAPE and call(maxp=129) == SHAPE
    assert call(maxo=129) == SHAPE and call(Hq=5) == SHAPE and call(mp=1 << 28, maxo=(1 << 30) + 1) == SHAPE
    assert call(Hq=2 ** 30, nq=1) == SHAPE
    for kw in (dict(D=96), dict(ps=24), dict(ps=8), dict(P=1 << 27), dict(B=4097), dict(groups=4097)):
        assert call(**kw) == UNSUPPORTED
    for x in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=x) == SCALE
    for n in ("q", "kp", "vp", "o", "ws"):
        assert call(**{n: MIS8}) == ALIGN
    assert call(ws=ctypes.c_void_p(A(20).value + 16)) == ALIGN
    for n in ("table", "lens", "starts", "pre", "lse"):
        assert call(**{n: MIS2}) == ALIGN
    assert call(ws=None) == WORKSPACE
    assert call(wsb=100) in (WORKSPACE, CUDA)
    for n in ("o", "lse"):
        for i in range(7):
            assert call(**{n: A(i)}) == ALIAS
    assert call(lse=A(7)) == ALIAS
    assert call() in (OK, CUDA) and call(lse=None, maxp=0, maxo=0) in (OK, CUDA)


def test_shared_decode_workspace_sizes(lib):
    size = lib.attn_paged_decode_shared_f16_workspace_size
    for bad in ((0, 4, 2, 1, 1, 64, 64, 128), (2, 5, 2, 1, 1, 64, 64, 128), (2, 4, 2, 1, 0, 64, 64, 128),
                (2, 4, 2, 1, 1, -1, 64, 128), (2, 4, 2, 1, 1, 64, -1, 128)):
        assert size(*bad) == 0
    # beside the ordinary decode's, a record of every row and 256 rows a CTA, and the tables
    plain = lib.attn_paged_decode_f16_workspace_size(64, 32, 8, 1, 2048, 128, 0)
    rows = 152 * 256 + 64 * 32
    extra = size(64, 32, 8, 1, 3, 1 << 20, 2048, 128) - plain
    assert rows * (128 * 4 + 8) <= extra <= rows * (128 * 4 + 8) + 64 * 8 + 200


def test_wrappers_refuse_wrong_arguments(lib):
    import torch
    import attention_fp16_flashattention_gb300 as gb
    z = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda x: gb.kv_paged_extend(x, i, i, i, i, 16, 4),
                 lambda x: gb.kv_paged_release(x, i, i, i, 16, 4),
                 lambda x: gb.qk_norm_rope_f16(x, None, i, z),
                 lambda x: gb.kv_paged_rope_append(x, z, z, i, z, z, i, z),
                 lambda x: gb.attn_paged_decode_shared_f16_fwd(x, z, z, i, i, i, i)):
        for x in (z, i, None):
            with pytest.raises(ValueError):
                call(x)


# ---------------------------------------------------------------- the oracles

def test_oracle_extend_by_hand():
    table = np.array([[4, -1, -1], [5, 6, -1], [-1, -1, -1]])
    out, lens, stack, tokens, refused = OT.extend(table, [15, 32, 0], [3, 1, 33], [9, 8, 7, 3], 16)
    # 15 + 3 takes one page (3), 32 + 1 one (7), 33 would take three of two
    assert out.tolist() == [[4, 3, -1], [5, 6, 7], [-1, -1, -1]] and lens == [18, 33, 0]
    assert stack == [9, 8] and refused == [2]
    assert tokens[0] == ([15, 16, 17], [4 * 16 + 15, 3 * 16, 3 * 16 + 1])
    assert tokens[1] == ([32], [7 * 16]) and tokens[2] == ([-1] * 33, [-1] * 33)
    pos, slots, starts = OT.packed(tokens, 5)
    assert pos.tolist() == [15, 16, 17, 32, -1] and starts.tolist() == [0, 3, 4, 37]
    assert OT.rows(tokens[:2], 3)[0].tolist() == [[15, 16, 17], [32, -1, -1]]
    # a sequence that needs no page is served behind one that gets none
    assert OT.extend(table, [15, 30], [40, 2], [1], 16)[1] == [15, 32]


def test_oracle_release_by_hand():
    table = np.array([[4, 3, -1], [5, 6, 7], [8, -1, -1]])
    assert OT.release(table, [18, 33, 16], [16, 17, 0], [9], 16, 20) == [9, 3, 7, 8]
    assert OT.release(table, [18, 33, 16], [0, 0, 0], [9], 16, 4) == [9, 4, 3]


def test_oracle_rotation_by_hand():
    x = np.zeros((1, 1, 1, 8))
    x[0, 0, 0] = [1, 2, 3, 4, 5, 6, 7, 8]
    f = np.array([np.pi / 2, np.pi])
    pos = np.array([[[1]]])
    y, size = OR.rotate(x, pos, f)                     # pairs (0, 2) by 90 degrees, (1, 3) by 180
    assert np.allclose(y[0, 0, 0], [-3, -2, 1, -4, 5, 6, 7, 8])
    assert size[0, 0, 0].tolist() == [4, 6, 4, 6, 5, 6, 7, 8]
    y, _ = OR.rotate(x, pos, f, interleaved=True, scale=2.0)
    assert np.allclose(y[0, 0, 0], [-4, 2, -6, -8, 5, 6, 7, 8])
    y, _ = OR.rotate(x, np.array([[[1]], [[3]]]), f, sections=[1, 1])
    assert np.allclose(y[0, 0, 0], [-3, -2, 1, -4, 5, 6, 7, 8])    # three half turns are one
    y, _ = OR.rotate(x, pos, None, weight=np.full(8, 3.0), eps=0.0)
    assert math.isclose((y * y).mean(), 9.0)
    # scores depend on the distance alone
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    f = 100.0 ** (-np.arange(32) / 32)
    dots = [float((OR.rotate(q, np.array([[[p + 7]]]), f)[0] * OR.rotate(k, np.array([[[p]]]), f)[0]).sum())
            for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0])


def test_frequencies_of_long_contexts():
    import attention_fp16_flashattention_gb300 as gb
    plain = gb.rope_frequencies(128, device="cpu").double().numpy()
    p = np.arange(64)
    assert np.allclose(plain, 10000.0 ** (-p / 64), rtol=2.0 ** -24)
    assert np.allclose(gb.rope_frequencies(128, factor=8, device="cpu"), plain / 8, rtol=1e-7)
    based = gb.rope_frequencies(128, factor=8, method="base", device="cpu").double().numpy()
    assert math.isclose(based[0], 1) and math.isclose(based[-1], plain[-1] / 8, rel_tol=1e-6)
    turns = 8192 * plain / (2 * np.pi)
    for method in ("turns", "pairs"):
        f = gb.rope_frequencies(128, 10000.0, 8, 8192, method, 1.0, 4.0, device="cpu").double().numpy()
        assert (np.diff(f) < 0).all()
        ratio = plain / f
        assert np.allclose(ratio[turns > 5], 1, rtol=1e-6) and np.allclose(ratio[turns < 0.8], 8, rtol=1e-6)
        assert ((ratio > 0.999) & (ratio < 8.001)).all()
        mid = ratio[(turns > 1.3) & (turns < 3.5)]
        assert len(mid) > 3 and ((mid > 1) & (mid < 8)).all()
    for bad in (dict(rot=7), dict(rot=64, base=1.0), dict(rot=64, factor=0), dict(rot=64, method="x"),
                dict(rot=64, method="turns"), dict(rot=2, method="base"),
                dict(rot=64, method="pairs", trained_len=9, low_turns=2, high_turns=1)):
        with pytest.raises(ValueError):
            gb.rope_frequencies(**dict(dict(rot=64, device="cpu"), **bad))
