"""K and V whose strides differ only where a dimension has one entry are laid out alike: one new
token per sequence, one KV head, one key."""

import numpy as np
import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def normal(*shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(shape))
    return torch.randn(shape, generator=g, device=DEV).half()


def test_append_one_token_of_two_layouts(gb):
    """K dense [B, H, 1, D], V a token-major projection seen as [B, H, 1, D]."""
    _, kp, vp, table, lens, _ = (torch.from_numpy(x).to(DEV) for x in
                                 inputs.paged_f16_inputs(3, 4, 4, 1, (5, 16, 17), 64, 3, page_size=16))
    k = normal(3, 4, 1, 64)
    v = normal(3, 4 * 64).view(3, 1, 4, 64).transpose(1, 2)
    assert k.stride() != v.stride() and k.shape == v.shape
    gb.kv_paged_append_f16(k, v, kp, vp, table, lens)
    assert gb.device_status() == 0
    for b, n in enumerate((5, 16, 17)):
        page, slot = table[b, (n - 1) // 16], (n - 1) % 16
        assert torch.equal(kp[page, slot], k[b, :, 0]) and torch.equal(vp[page, slot], v[b, :, 0])


@pytest.mark.parametrize("Hkv,Skv", [(1, 70), (2, 1)])
def test_diff_prompt_of_two_layouts(gb, Hkv, Skv):
    """K head-major, V token-major, which is one layout where there is one head or one key."""
    q = normal(2, 2, 40, 128)
    k = normal(2, Hkv, Skv, 128)
    v = normal(2, Skv, Hkv, 128).transpose(1, 2)
    assert k.stride() != v.stride()
    vecs, weight = (torch.from_numpy(x).to(DEV) for x in inputs.diff_inputs(2, 128, 4))
    o = gb.attn_diff_prefill_fwd(q, k, v, vecs, 0.5, weight, causal=False)
    want = gb.attn_diff_prefill_fwd(q, k, v.clone(memory_format=torch.contiguous_format), vecs, 0.5,
                                    weight, causal=False)
    assert torch.equal(o, want) and gb.device_status() == 0


def test_layouts_that_differ_are_refused(gb):
    q, k, v = normal(2, 2, 9, 128), normal(2, 2, 9, 128), normal(2, 9, 2, 128).transpose(1, 2)
    vecs = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError, match="strides"):
        gb.attn_diff_prefill_fwd(q, k, v, vecs, 0.5)
    pages = torch.zeros((2, 16, 2, 128), dtype=torch.float16, device=DEV)
    table, lens = (torch.from_numpy(np.array(x, dtype=np.int32)).to(DEV) for x in ([[0], [1]], [9, 9]))
    with pytest.raises(ValueError, match="strides"):
        gb.kv_paged_append_f16(k, v, pages, pages.clone(), table, lens)
