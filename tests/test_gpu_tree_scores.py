"""GPU tests of tg_tree_attention where scores are large: a common offset that takes the
logits to where fp32 has steps of 4 to 16 (the weights' range must hold there)."""
import pytest
import torch

from test_gpu_tree_attn import BF, E4, I8, api, make, run, _status  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("T,hq,hkv,dh", [(2, 16, 8, 128), (1, 8, 8, 64), (8, 16, 8, 128), (8, 16, 8, 64), (20, 16, 8, 128)])
@pytest.mark.parametrize("base,ahead", [(2.0 ** 24.5, 4), (5.8e7, 8), (9.0e7, 8), (1.1e8, 16), (1.7e8, 16), (2.5e8, 32)])
def test_keys_one_step_ahead_on_a_large_offset(api, fmt, T, hq, hkv, dh, base, ahead):
    # Every 32 keys two count: the first (value A) and the 17th (value B), whose score is
    # `ahead` higher, so that its logit of gain 1 is 1.44 x ahead higher in units of log2. fp32
    # logits there have steps of `ahead` or less, and the rounding of both takes at most one step:
    # what is left is more than 0.44 x ahead and a multiple of the step, so at least ahead / 2, and
    # A weighs at most 2^-(ahead / 2) of B. All others weigh nothing.
    n = 512
    for off in range(0, 10):
        st = make(3, 1, T, n, [n], hq, hkv, dh, fmt, garbage=False)
        s0 = torch.tensor(base).double().div(ahead).floor().add(off).mul(ahead).float()
        assert float(s0 + ahead) - float(s0) == ahead
        st["gain"].fill_(1.0)
        st["q"].zero_()
        st["mask"].zero_()
        st["sc"].zero_()
        st["sc"][0, 0::32] = s0.cuda()
        st["sc"][0, 16::32] = (s0 + ahead).cuda()
        a, b = 3.0, -5.0
        v = torch.zeros(n)
        v[0::32], v[16::32] = a, b
        st["vc"][0] = v[:, None, None].expand(n, hkv, dh).to(BF).to(fmt).cuda()
        if st["vs"] is not None:
            st["vs"].fill_(1.0)
        got = run(api, st).double()
        assert torch.isfinite(got).all(), (off, float(s0))
        # the output's rounding, the weight's, and A's part
        tol = abs(b) * (2.0 ** -8 + 2.0 ** -11) + (a - b) * 2.0 ** -(ahead // 2)
        assert ((got - b).abs() <= tol).all(), (off, float((got - b).abs().max()), tol)
