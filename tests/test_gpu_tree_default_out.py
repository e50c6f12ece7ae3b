"""GPU test of tg_tree_attention's binding without an output of the caller's: rows behind
each sequence's drafts, and those of a sequence that is skipped, are zeros and not what
the allocator's block held before."""
import pytest
import torch

from test_gpu_tree_attn import BF, I8, api, check, make, reference, run  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [BF, I8])
@pytest.mark.parametrize("other_stream", [False, True])
def test_rows_that_are_not_drafted_are_zeros(api, fmt, other_stream):
    st = make(17, 3, 6, 50, [50, 20, 0], 4, 2, 128, fmt, dls=[6, 2, 0])
    stream = torch.cuda.Stream() if other_stream else None
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):   # the blocks that the call will get hold NaN
        old = [torch.full_like(st["q"], float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        del old
    out = run(api, st, stream=stream)
    torch.cuda.synchronize()
    check(out, reference(st), keep=0.0)
    st["len"][0] = -1
    out = run(api, st, stream=stream, max_len=50)
    torch.cuda.synchronize()
    assert api.device_status(reset=True) == 7
    assert (out[0] == 0).all() and (out[2] == 0).all()
