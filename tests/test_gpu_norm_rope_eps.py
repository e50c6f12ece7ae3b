"""GPU tests of tg_qk_norm_rope and its backward without an epsilon: eps = 0 is a valid
call, and heads that a lane group has no work for must not enter the weight gradients
(1 / sqrt(0) there is infinite). Inputs, tolerances and their derivation are those of
test_gpu_norm_rope.py; with eps = 0 the mean has one rounding less."""
import pytest
import torch

import ops_ref
from test_gpu_norm_rope import U, _check_fwd, _close, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from learned_token_pruning_gemm_b200 import api, build
    build.build()
    api.device_status(reset=True)
    return api


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,hq,hkv,dh,rot", [
    (1, 16, 8, 128, 128),      # few tokens: warps share one, most lane groups lack a head in some round
    (1, 1, 1, 8, 8),
    (7, 3, 1, 96, 96),
    (333, 2, 1, 128, 128),     # fewer heads than a warp takes at once
    (333, 5, 2, 64, 32),
    (2500, 4, 2, 128, 64),     # a warp a token, and more tokens than warps
    (130, 8, 2, 256, 64),
])
def test_no_epsilon(api, T, hq, hkv, dh, rot, dt):
    q, k, wq, wk, pos, dq, dk = _inputs(T + dh + 3, T, hq, hkv, dh, dt, False)
    _check_fwd(api.qk_norm_rope(q, k, wq, wk, pos, eps=0.0, rope_base=1e4, rot_dim=rot), q, k, wq, wk, pos, rot, 1e4, 0.0)
    got = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, eps=0.0, rope_base=1e4, rot_dim=rot)
    cos, sin = ops_ref.rotation(pos, rot, 1e4)
    fp = 32 * U if dt == torch.float32 else 2.0 ** -19
    for i, (x, w, dy, name) in enumerate(((q, wq, dq, "dq"), (k, wk, dk, "dk"))):
        dx, dw, size, dw_size = ops_ref.norm_rope_bwd(x, w, cos, sin, 0.0, dy)
        _close(got[i], dx, (torch.finfo(dt).eps / 2) * dx.abs() * (1 + 2.0 ** -7) + fp * size + 1e-37, name)
        _close(got[2 + i], dw, (64 * U + fp) * dw_size + 1e-37, name + "_weight")
    assert api.device_status(reset=True) == 0
