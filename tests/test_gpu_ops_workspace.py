"""GPU tests that workspaces need no initial value: calls over ones filled with NaN bit
patterns, and over what a call of another shape left in them, give the bits of a call over
zeros."""
import pytest
import torch

import test_gpu_norm_rope
from test_gpu_tree_attn import BF, CASES, E4, EDGES, I8, api, make, run, _status  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_tree_attention(api, fmt):
    calls = []
    for i, (B, T, cap, lens, hq, hkv, dh, dls) in enumerate(CASES + EDGES):
        st = make(50 + i, B, T, cap, lens, hq, hkv, dh, fmt, dls)
        for ml in {max(lens), cap}:
            calls.append((st, ml, max(16, api.tree_attention_workspace_size(B, T, hq, hkv, dh, ml))))
    left = torch.zeros(max(n for _, _, n in calls), dtype=torch.uint8, device="cuda")
    for st, ml, n in calls:
        outs = []
        for ws in (torch.zeros(n, dtype=torch.uint8, device="cuda"),
                   torch.full((n,), 255, dtype=torch.uint8, device="cuda"), left):
            outs.append(run(api, st, out=torch.full_like(st["q"], 9.0), max_len=ml, workspace=ws))
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_norm_backward(api, dt):
    left = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    for T, hq, hkv, dh in ((1, 16, 8, 128), (5000, 4, 2, 64), (77, 3, 1, 40), (600, 8, 8, 256)):
        q, k, wq, wk, pos, dq, dk = test_gpu_norm_rope._inputs(T, T, hq, hkv, dh, dt, False)
        n = api.qk_norm_rope_bwd_workspace_size(T, hq, hkv, dh)
        outs = [api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, workspace=ws)
                for ws in (torch.zeros(n, dtype=torch.uint8, device="cuda"),
                           torch.full((n,), 255, dtype=torch.uint8, device="cuda"), left)]
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(outs[0], o))
