"""GPU tests of tg_tree_attention at the ends of its sizes: the largest batch (whose
sequence table is the most that the kernels' shared memory holds), batches that grow, and
the widest group with the most drafted tokens. Tolerances as in test_gpu_tree_attn.py."""
import pytest
import torch

from test_gpu_tree_attn import BF, E4, I8, api, check, make, reference, run, _status  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, I8])
@pytest.mark.parametrize("T,hq,hkv,dh", [(1, 2, 2, 128), (2, 8, 1, 64), (20, 2, 2, 64)])
def test_largest_batch(api, fmt, T, hq, hkv, dh):
    B = 1024
    lens = [(37 * b) % 23 for b in range(B)]
    dls = [1 + (b % T) if b % 5 else T for b in range(B)] if T < 20 else [(b * 7) % 3 for b in range(B)]
    st = make(23, B, T, 24, lens, hq, hkv, dh, fmt, dls)
    check(run(api, st, out=torch.full_like(st["q"], 9.0)), reference(st))


def test_batches_that_grow(api):
    # one sequence after the other joins; what was there stays as it was
    B = 40
    st = make(24, B, 1, 70, [(31 * b) % 71 for b in range(B)], 8, 8, 128, E4)
    whole = run(api, st, max_len=70)
    ref = reference(st)
    check(whole, ref, keep=None)
    for n in range(1, B + 1):
        part = {k: t if t is None or k in ("gain", "tau") else t[:n] for k, t in st.items()}
        check(run(api, part, max_len=70), (ref[0][:n], ref[1][:n]), keep=None)


@pytest.mark.parametrize("fmt", [BF, I8])
@pytest.mark.parametrize("T,hq,hkv,dh", [(64, 128, 1, 64), (64, 65, 1, 128), (33, 192, 3, 64)])
def test_widest_groups(api, fmt, T, hq, hkv, dh):
    st = make(25, 1, T, 200, [197], hq, hkv, dh, fmt, [T - 1])
    check(run(api, st, out=torch.full_like(st["q"], 9.0)), reference(st))
