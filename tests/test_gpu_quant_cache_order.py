"""GPU tests of the quantised cache for offsets that do not ascend. Two sequences may then
claim the same packed rows: each sequence is written whole, with its new length, or left
as it was, with its old one, and the call is recorded; the same for what is given back."""
import pytest
import torch

import ops_ref
from test_gpu_quant_cache import _append, _empty, _rows, _same, api  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
CHECK = 7


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _run(api, cu, cap, R, start, in_place, hkv=1, dh=64):
    """Appends and reads back; returns the sequences that were written. Checks that each was
    written whole or not at all, and that no packed row went to two."""
    B = len(cu) - 1
    k, v, s = _rows(2, R, hkv, dh)
    c = _empty(B, cap, hkv, dh, torch.int8)
    before = {n: t.clone() for n, t in c.items()}
    ln = _i32(start) if in_place else _i32([cap - 1] * B)
    old = ln.tolist()
    _append(api, c, ln, k, v, s, _i32(cu), start=None if in_place else _i32(start))
    assert api.device_status(reset=True) == CHECK
    now, before = {n: t.cpu() for n, t in c.items()}, {n: t.cpu() for n, t in before.items()}
    stored = {"sc": s.cpu()}
    for name, x in (("k", k), ("v", v)):
        q, stored[name + "s"] = (t.cpu() for t in ops_ref.quantise(x, torch.int8))
        stored[name + "c"] = q.to(torch.int8)
    written, taken, want = [], set(), {n: t.clone() for n, t in before.items()}
    for b, new in enumerate(ln.tolist()):
        n, r, at = cu[b + 1] - cu[b], slice(cu[b], cu[b + 1]), slice(start[b], start[b] + cu[b + 1] - cu[b])
        if n <= 0:
            assert new in ((old[b], start[b]) if n == 0 else (old[b],)), b
        elif not torch.equal(now["sc"][b], before["sc"][b]):
            assert cu[b] >= 0 and cu[b + 1] <= R and new == start[b] + n, b
            rows = set(range(cu[b], cu[b + 1]))
            assert not rows & taken
            taken |= rows
            written.append(b)
            for name in want:
                want[name][b, at] = stored[name][r]
        else:
            assert new == old[b], b
    _same(now, want)
    out = (torch.full((R, hkv, dh), 9.0).cuda(), torch.full((R, hkv, dh), 9.0).cuda(), torch.full((R,), 9.0).cuda())
    api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], _i32([cap] * B), _i32(cu), R, out=out, start=_i32(start))
    assert api.device_status(reset=True) == CHECK
    scores = out[2].cpu()
    for b in written:
        assert torch.equal(scores[cu[b]:cu[b + 1]], stored["sc"][cu[b]:cu[b + 1]])
    rest = torch.ones(R, dtype=torch.bool)
    rest[sorted(taken)] = False
    assert (scores[rest] == 9).all() and (out[0].cpu()[rest] == 9).all()
    return written


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("cu", [[0, 10, 5, 8], [0, 5, 3, 10], [0, 3, 3, 2], [4, 3, 3, 10], [0, 10, 10, -1], [0, 4, 2, 7, 5, 9, 9, 1],
                                [9, 8, 7, 6, 5, 4, 3, 2, 1, 0], [0, 9, 1, 9, 1, 9, 1, 9]])
def test_overlapping_sequences(api, cu, in_place):
    _run(api, cu, 20, 10, [(3 * b) % 5 for b in range(len(cu) - 1)], in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B", [40, 1024, 1025, 2500])
@pytest.mark.parametrize("at", [0.01, 0.5, 1])
def test_one_offset_among_many(api, B, at, in_place):
    # the offsets of many sequences, one of them out of order by a little or by much
    i = max(1, int(at * (B - 1)))
    for by in (1, 7, -B):
        cu = [2 * b for b in range(B + 1)]
        cu[i] = max(0, cu[i + 1] + by)
        written = _run(api, cu, 4, 2 * B, [b % 3 for b in range(B)], in_place)
        assert len(written) < B


@pytest.mark.parametrize("B", [5, 300, 1500])
def test_random_offsets(api, B):
    g = torch.Generator().manual_seed(B)
    for _ in range(6):
        cu = torch.randint(0, 3 * B, (B + 1,), generator=g)
        cu = torch.where(torch.rand(B + 1, generator=g) < 0.8, torch.sort(cu).values, cu)
        if (cu[1:] >= cu[:-1]).all():
            continue
        _run(api, cu.tolist(), 40, 3 * B, [0] * B, bool(B % 2))
