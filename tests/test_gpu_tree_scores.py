"""GPU tests of tg_tree_attention where scores are large: a common offset that takes the
logits to where fp32 has steps of 4 to 16 (the weights' range must hold there), and
scores of the type's lowest value (finite: a row of them is a mean, not a row of nothing)."""
import pytest
import torch

from test_gpu_tree_attn import BF, E4, I8, api, check, make, reference, run, values, _status  # noqa: F401 (fixtures)

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


LOWEST, HIGHEST = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
SHAPES = [(1, 4, 2, 128), (3, 8, 4, 64), (20, 8, 2, 128), (64, 8, 2, 64)]   # T, hq, hkv, dh


@pytest.mark.parametrize("score", [LOWEST, HIGHEST, -3e38, 2.0 ** 121])
@pytest.mark.parametrize("gain", [0.25, 1.0, 7.0, 80.0])
@pytest.mark.parametrize("fmt", [BF, I8])
def test_a_token_alone_is_its_value_whatever_its_score(api, fmt, gain, score):
    # over an empty cache, and over one whose rows weigh nothing: the weight is 1 exactly
    for n in (0, 300):
        st = make(12, 2, 3, 300, [n, n], 4, 2, 128, fmt, garbage=False)
        st["gain"].fill_(gain)
        st["sd"].fill_(score)
        st["sc"].fill_(float("-inf"))
        st["mask"].copy_(torch.tensor([1, 2, 4]).cuda())
        assert torch.equal(run(api, st, max_len=300), st["vd"].repeat_interleave(2, 2))


@pytest.mark.parametrize("score", [LOWEST, HIGHEST])
@pytest.mark.parametrize("T,hq,hkv,dh", SHAPES)
@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_rows_of_nothing_but_lowest_scores(api, fmt, T, hq, hkv, dh, score):
    # All logits are equal (in 64 bits too: what q and k add is below their last place). Over codes the value
    # scales' part of the weights is below it as well, so there the output is only known
    # to lie within the values.
    st = make(13, 2, T, 400, [400, 77], hq, hkv, dh, fmt, garbage=False)
    st["gain"].add_(0.3)
    st["sc"].fill_(score)
    st["sd"].fill_(score)
    got = run(api, st)
    if fmt == BF:
        check(got, reference(st))
    v = torch.cat([values(st)[1], st["vd"].double()], 1)
    for b, n in enumerate((400, 77)):
        rows = torch.cat([v[b, :n], v[b, 400:]])
        lo, hi = (f(rows, 0).repeat_interleave(hq // hkv, 0) for f in (torch.amin, torch.amax))
        assert (got[b] >= lo - 2.0 ** -8 * lo.abs()).all() and (got[b] <= hi + 2.0 ** -8 * hi.abs()).all()
    # next to others they weigh nothing, or everything
    st["sc"][:, 5:30] = 0.5
    st["sd"].fill_(-0.5)
    if fmt == BF or score == LOWEST:
        check(run(api, st), reference(st))
    # and minus infinity weighs nothing next to them
    st["sc"].fill_(float("-inf"))
    st["sc"][:, 11] = score
    st["sd"].fill_(float("-inf"))
    check(run(api, st), reference(st))
