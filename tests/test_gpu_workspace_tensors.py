"""What the calls on paged FP16 caches and differential prompts take for a workspace: a tensor whose
bytes are all its own.  Each refusal comes before anything is queued."""

import pytest
import torch

from attention_fp16_flashattention_gb300 import inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("call", ["decode", "diff decode", "diff prompt"])
def test_workspaces_that_are_refused(gb, call):
    q, kp, vp, table, lens, _ = (torch.from_numpy(x).to(DEV) for x in
                                 inputs.paged_f16_inputs(2, 4, 2, 1, (40, 9000), 128, 95))
    vecs, _ = inputs.diff_inputs(4, 128, 96)
    vecs = torch.from_numpy(vecs).to(DEV)
    kv = torch.zeros((2, 2, 9000, 128), dtype=torch.float16, device=DEV)
    run = {"decode": lambda ws: gb.attn_paged_decode_f16_fwd(q, kp, vp, table, lens, workspace=ws),
           "diff decode": lambda ws: gb.attn_diff_paged_decode_f16_fwd(q, kp, vp, table, lens, vecs, 0.5,
                                                                       workspace=ws),
           "diff prompt": lambda ws: gb.attn_diff_prefill_fwd(q, kv, kv, vecs, 0.5, workspace=ws)}[call]
    n = {"decode": gb.attn_paged_decode_f16_workspace_size(2, 4, 2, 1, 9024, 128),
         "diff decode": gb.attn_diff_paged_decode_f16_workspace_size(2, 4, 2, 1, 9024, 128),
         "diff prompt": gb.attn_diff_prefill_workspace_size(2, 4, 1, 9000, 128)}[call]
    assert n > 1 << 10
    one = torch.empty(16, dtype=torch.uint8, device=DEV)
    for wrong in (one[:1].expand(n), one.view(1, 16).expand(n // 16 + 1, 16),
                  torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2],
                  torch.empty(n, dtype=torch.uint8), b"x" * 64):
        with pytest.raises(ValueError, match="workspace"):
            run(wrong)
    full = run(torch.empty(n, dtype=torch.uint8, device=DEV))
    words = run(torch.empty((n // 64 + 1, 16), dtype=torch.float32, device=DEV))   # any type and shape
    assert torch.equal(full, words) and gb.device_status() == 0
