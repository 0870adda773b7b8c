"""Refusals of the FP16 page cache and the differential calls (CPU only): arguments are checked
before any CUDA call, so placeholder addresses reach every branch; valid arguments end in
GBATTN_ERR_CUDA where no GPU is visible."""

import ctypes
import shutil
import os

import pytest

OK, NULL, SHAPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE, CUDA, SCALE = range(9)


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only validation tests: they run where no GPU is visible")
    from attention_fp16_flashattention_gb300 import build
    build.build()
    import attention_fp16_flashattention_gb300 as gb
    return gb.load()


def A(i):
    """Placeholder device addresses, 256 MiB apart, never dereferenced."""
    return ctypes.c_void_p(0x10000000 * (i + 1))


MIS8, MIS2 = ctypes.c_void_p(0x10000000 * 40 + 8), ctypes.c_void_p(0x10000000 * 41 + 2)


def caller(fn, names, base):
    def call(**kw):
        assert set(kw) <= set(names)
        return fn(*[kw.get(n, base[n]) for n in names])
    return call


def test_append_refusals(lib):
    names = ("k", "v", "kp", "vp", "table", "lens", "new", "w", "B", "Hkv", "n", "D", "st", "P",
             "ps", "mp", "stream")
    base = dict(zip(names, (A(0), A(1), A(2), A(3), A(4), A(5), A(6), A(7), 2, 2, 3, 128, None, 8,
                            16, 4, None)))
    call = caller(lib.kv_paged_append_f16, names, base)
    for n in ("k", "v", "kp", "vp", "table", "lens"):
        assert call(**{n: None}) == NULL
    for n in ("B", "Hkv", "n", "P", "ps", "mp"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(B=65536) == SHAPE
    for d in (0, 96, 512):
        assert call(D=d) == UNSUPPORTED
    for ps in (8, 24, 48):
        assert call(ps=ps) == UNSUPPORTED
    assert call(P=1 << 27, ps=16) == UNSUPPORTED          # slots pass 31 bits
    st = (ctypes.c_int64 * 3)(1, 2, 3)
    assert call(st=st) == SHAPE
    assert call(k=MIS8) == ALIGN and call(vp=MIS8) == ALIGN and call(table=MIS2) == ALIGN
    assert call(w=MIS2) == ALIGN and call(new=MIS2) == ALIGN
    assert call(k=A(2)) == ALIAS and call(vp=A(2)) == ALIAS and call(w=A(3)) == ALIAS
    assert call(lens=A(7)) == ALIAS
    assert call() in (OK, CUDA) and call(new=None, w=None) in (OK, CUDA)
    packed = (ctypes.c_int64 * 3)(3 * 2 * 128, 128, 2 * 128)
    assert call(st=packed) in (OK, CUDA)


DEC = ("q", "kp", "vp", "table", "lens", "o", "lse", "w", "B", "Hq", "Hkv", "nq", "D", "P", "ps",
       "mp", "max", "scale", "ws", "wsb", "stream")
DIFF = ("q", "kp", "vp", "table", "lens", "vecs", "heads", "init", "norm", "eps", "o", "lse", "B",
        "Hq", "Hkv", "nq", "D", "P", "ps", "mp", "max", "scale", "ws", "wsb", "stream")


@pytest.mark.parametrize("diff", [False, True])
def test_decode_refusals(lib, diff):
    common = dict(q=A(0), kp=A(1), vp=A(2), table=A(3), lens=A(4), o=A(5), lse=A(6), B=2, Hq=4,
                  Hkv=2, nq=1, D=128, P=8, ps=16, mp=4, max=64, scale=0.1, ws=A(8), wsb=1 << 27,
                  stream=None)
    if diff:
        call = caller(lib.attn_diff_paged_decode_f16_fwd, DIFF,
                      dict(common, vecs=A(9), heads=4, init=0.5, norm=A(10), eps=1e-5))
    else:
        call = caller(lib.attn_paged_decode_f16_fwd, DEC, dict(common, w=A(7)))
    for n in ("q", "kp", "vp", "table", "lens", "o"):
        assert call(**{n: None}) == NULL
    for n in ("B", "Hq", "Hkv", "nq", "P", "ps", "mp", "max"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -3}) == SHAPE
    assert call(Hq=5) == SHAPE and call(max=65) == SHAPE
    assert call(mp=1 << 28, max=(1 << 30) + 1) == SHAPE
    for d in (0, 32, 96, 512) + ((64, 256) if diff else ()):
        assert call(D=d) == UNSUPPORTED
    for ps in (8, 24):
        assert call(ps=ps, max=16) == UNSUPPORTED
    assert call(P=1 << 27) == UNSUPPORTED and call(B=4097) == UNSUPPORTED
    assert call(Hq=2 ** 31 - 2, nq=2 ** 30) == SHAPE       # rows pass 31 bits
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == SCALE
    for n in ("q", "kp", "vp", "o", "ws"):
        assert call(**{n: MIS8}) == ALIGN
    for n in ("table", "lens", "lse"):
        assert call(**{n: MIS2}) == ALIGN
    assert call(o=A(0)) == ALIAS and call(lse=A(1)) == ALIAS and call(lse=A(5)) == ALIAS
    assert call(ws=None) == WORKSPACE
    assert call(lse=None) in (OK, CUDA) and call() in (OK, CUDA)
    if diff:
        assert call(vecs=None) == NULL and call(heads=2) == SHAPE and call(heads=0) == SHAPE
        assert call(init=float("nan")) == SCALE and call(init=float("inf")) == SCALE
        assert call(eps=0.0) == SCALE and call(eps=float("nan")) == SCALE
        assert call(norm=None, eps=0.0) in (OK, CUDA) and call(heads=1) in (OK, CUDA)
        assert call(vecs=MIS2) == ALIGN and call(norm=MIS2) == ALIGN
        assert call(o=A(9)) == ALIAS and call(lse=A(10)) == ALIAS
    else:
        assert call(w=MIS2) == ALIGN and call(w=A(2)) == ALIAS and call(w=A(5)) == ALIAS
        assert call(w=None) in (OK, CUDA)


def test_decode_workspace_sizes(lib):
    plain = lib.attn_paged_decode_f16_workspace_size
    assert plain(0, 4, 2, 1, 64, 128, 0) == 0 and plain(2, 5, 2, 1, 64, 128, 0) == 0
    base = plain(2, 4, 2, 1, 4096, 128, 0)
    # with weights: a (max, 1 / sum) pair per row, 16 bytes per tile, a score per row and token
    assert plain(2, 4, 2, 1, 4096, 128, 1) == base + 2 * 4 * 8 + 2 * 2 * 256 * 16 + 2 * 4 * 4096 * 4
    assert lib.attn_diff_paged_decode_f16_workspace_size(2, 4, 2, 1, 4096, 128) == base
    assert plain(4096, 64, 8, 1, 1 << 20, 128, 1) > 1 << 40      # no 32-bit wrap


def test_evict_refusals(lib):
    names = ("kp", "vp", "w", "table", "dst", "lens", "new", "kept", "B", "Hkv", "D", "elem", "P",
             "ps", "mp", "dp", "max", "budget", "sink", "recent", "stream")
    base = dict(zip(names, (A(0), A(1), A(2), A(3), A(4), A(5), A(6), A(7), 2, 2, 128, 2, 8, 16, 4,
                            2, 64, 32, 2, 4, None)))
    call = caller(lib.kv_paged_evict, names, base)
    for n in ("kp", "vp", "w", "table", "dst", "lens", "new", "kept"):
        assert call(**{n: None}) == NULL
    for n in ("B", "Hkv", "P", "ps", "mp", "dp", "max", "budget"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(sink=-1) == SHAPE and call(recent=-1) == SHAPE
    assert call(sink=20, recent=13) == SHAPE and call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == SHAPE
    assert call(max=65) == SHAPE and call(budget=33) == SHAPE      # past the pages
    assert call(dst=A(3)) == SHAPE and call(dst=A(3), dp=4) in (OK, CUDA)
    for d, e in ((96, 2), (128, 4), (512, 1), (32, 2)):
        assert call(D=d, elem=e) == UNSUPPORTED
    assert call(ps=24) == UNSUPPORTED and call(P=1 << 27) == UNSUPPORTED
    for n in ("kp", "vp"):
        assert call(**{n: MIS8}) == ALIGN
    for n in ("w", "table", "dst", "lens", "new", "kept"):
        assert call(**{n: MIS2}) == ALIGN
    assert call(vp=A(0)) == ALIAS and call(new=A(5)) == ALIAS and call(kept=A(6)) == ALIAS
    assert call(w=A(0)) == ALIAS and call(kept=A(3)) == ALIAS
    assert call(elem=1) in (OK, CUDA) and call() in (OK, CUDA)


def test_diff_prefill_refusals(lib):
    names = ("q", "k", "v", "vecs", "heads", "init", "norm", "eps", "ql", "kl", "o", "lse", "B",
             "Hq", "Hkv", "Sq", "Skv", "D", "qs", "ks", "os", "scale", "causal", "ws", "wsb",
             "stream")
    base = dict(zip(names, (A(0), A(1), A(2), A(3), 4, 0.5, A(4), 1e-5, A(5), A(6), A(7), A(8), 2, 4,
                            2, 100, 200, 128, None, None, None, 0.125, 1, None, 0, None)))
    call = caller(lib.attn_diff_prefill_fwd, names, base)
    for n in ("q", "k", "v", "vecs", "o"):
        assert call(**{n: None}) == NULL
    for n in ("B", "Hq", "Hkv", "Sq", "Skv"):
        assert call(**{n: 0}) == SHAPE and call(**{n: -1}) == SHAPE
    assert call(Hq=5) == SHAPE and call(heads=3) == SHAPE and call(causal=2) == SHAPE
    assert call(B=65536) == SHAPE and call(Sq=(1 << 22) + 1) == SHAPE
    assert call(Skv=(1 << 30) + 1) == SHAPE
    for d in (64, 256, 0):
        assert call(D=d) == UNSUPPORTED
    st = (ctypes.c_int64 * 3)(1, 2, 3)
    assert call(qs=st) == SHAPE and call(ks=st) == SHAPE and call(os=st) == SHAPE
    assert call(os=(ctypes.c_int64 * 3)(0, 128, 128)) == SHAPE          # output heads overlap
    for s in (0.0, float("nan"), float("inf")):
        assert call(scale=s) == SCALE and call(eps=s) == SCALE
    assert call(init=float("nan")) == SCALE
    for n in ("q", "k", "v", "o", "ws"):
        assert call(**{n: MIS8}) == ALIGN
    for n in ("vecs", "norm", "ql", "kl", "lse"):
        assert call(**{n: MIS2}) == ALIGN
    assert call(o=A(1)) == ALIAS and call(lse=A(4)) == ALIAS and call(lse=A(7)) == ALIAS
    n = lib.attn_diff_prefill_workspace_size(2, 4, 100, 20000, 128)
    assert n > 0 and call(Skv=20000, ws=A(0), wsb=n) == ALIAS           # a workspace that is used
    assert call(ql=None, kl=None, lse=None, norm=None, eps=0.0) in (OK, CUDA)
    assert call() in (OK, CUDA)
    assert lib.attn_diff_prefill_workspace_size(1, 16, 8192, 8192, 128) == 0     # enough rows


def test_wrappers_refuse_cpu_tensors(lib):
    import torch
    import attention_fp16_flashattention_gb300 as gb
    z = torch.zeros(1, 1, 1, 64, dtype=torch.float16)
    for call in (lambda x: gb.kv_paged_append_f16(x, z, z, z, z, z),
                 lambda x: gb.attn_paged_decode_f16_fwd(x, z, z, z, z),
                 lambda x: gb.kv_paged_evict(x, z, z, z, z, 4),
                 lambda x: gb.attn_diff_paged_decode_f16_fwd(x, z, z, z, z, z, 0.5),
                 lambda x: gb.attn_diff_prefill_fwd(x, z, z, z, 0.5)):
        for x in (z, None):
            with pytest.raises(ValueError):
                call(x)
