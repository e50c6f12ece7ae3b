"""GPU parity of tg_qk_norm_rope and its backward against the 64-bit forms of
ops_ref.py, through the binding.

Tolerances, per element. A stored value is off by half a step (torch.finfo(t).eps / 2
relative). Before that, in fp32 (u = 2^-24): the mean of squares takes at most 8 fused
sums a lane, 5 across lanes and one for eps (14 u, of which 7 u reach its root), the
root 1 u, the products x r w 2 u, the rotation 2 u and the sine and cosine 2 u plus the
angle's pi/4 u: below 16 u of |n_i| + |n_pair|. The 16-bit path takes MUFU sines, off by
at most 2^-21 for angles up to pi: 2^-20 of the pair's size with room for the product.
Backward: the same errors in g and r, and the mean over the head once more: 32 u (fp32)
or 2^-19 (bf16) of the terms' size as ops_ref gives it. Weight gradients: at most 64
sequential fp32 sums per chain here (a lane's heads, then lanes, warps and blocks): 64 u
plus the terms' own 32 u or 2^-19."""
import numpy as np
import pytest
import torch

import ops_ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def api():
    from learned_token_pruning_gemm_b200 import api, build
    build.build()
    api.device_status(reset=True)
    return api


@pytest.fixture(autouse=True)
def _no_device_errors(api):
    yield
    assert api.device_status(reset=True) == 0, "a kernel recorded a device-side error"


def _inputs(seed, T, hq, hkv, dh, dt, packed, far=False):
    g = torch.Generator().manual_seed(seed)
    if packed:   # views of a packed projection output
        qkv = (torch.randn(T, hq + 2 * hkv, dh, generator=g) * 1.7).to(dt).cuda()
        q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]
    else:
        q = (torch.randn(T, hq, dh, generator=g) * 1.7).to(dt).cuda()
        k = (torch.randn(T, hkv, dh, generator=g) * 0.3).to(dt).cuda()
    wq, wk = (0.5 + torch.rand(dh, generator=g)).cuda(), (torch.rand(dh, generator=g) - 0.5).cuda()
    pos = torch.randint(0, 2 ** 31 - 1 if far else 40000, (T,), generator=g).to(torch.int32).cuda()
    pos[0] = 0
    dq = torch.randn(T, hq, dh, generator=g).to(dt).cuda()
    dk = torch.randn(T, hkv, dh, generator=g).to(dt).cuda()
    return q, k, wq, wk, pos, dq, dk


def _close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float(((got - want).abs() / tol.clamp_min(1e-300)).max()):.2f} of the tolerance")


def _check_fwd(out, q, k, wq, wk, pos, rot, base, eps):
    dt = q.dtype
    cos, sin = ops_ref.rotation(pos, rot, base)
    fp = 16 * U if dt == torch.float32 else 2.0 ** -20
    for got, x, w, name in ((out[0], q, wq, "q"), (out[1], k, wk, "k")):
        want = ops_ref.norm_rope(x, w, cos, sin, eps)
        n = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + eps) * w.double()
        tol = (torch.finfo(dt).eps / 2) * want.abs() * (1 + 2.0 ** -7) + fp * ops_ref.pair_size(n, cos)
        _close(got, want, tol + 1e-37, name)


CASES = [  # T, hq, hkv, dh, rot, dtype, packed
    (1, 16, 8, 128, 128, torch.bfloat16, True),
    (7, 16, 8, 128, 128, torch.bfloat16, False),
    (333, 4, 2, 64, 64, torch.bfloat16, True),
    (65, 5, 1, 96, 96, torch.bfloat16, False),
    (130, 8, 2, 256, 64, torch.bfloat16, True),
    (50, 3, 3, 24, 16, torch.bfloat16, False),
    (1, 1, 1, 8, 8, torch.float32, False),
    (33, 6, 2, 128, 32, torch.float32, True),
    (257, 8, 2, 256, 256, torch.float32, False),
    (20, 2, 1, 40, 0, torch.float32, True),
    (6000, 3, 1, 64, 48, torch.bfloat16, True),   # more tokens than warps
]


@pytest.mark.parametrize("T,hq,hkv,dh,rot,dt,packed", CASES)
def test_forward(api, T, hq, hkv, dh, rot, dt, packed):
    q, k, wq, wk, pos, _, _ = _inputs(T + dh, T, hq, hkv, dh, dt, packed, far=T < 100)
    out = api.qk_norm_rope(q, k, wq, wk, pos, eps=1e-6, rope_base=1e6, rot_dim=rot)
    _check_fwd(out, q, k, wq, wk, pos, rot, 1e6, float(np.float32(1e-6)))


@pytest.mark.parametrize("T,hq,hkv,dh,rot,dt,packed", CASES)
def test_backward(api, T, hq, hkv, dh, rot, dt, packed):
    q, k, wq, wk, pos, dq, dk = _inputs(T + dh + 1, T, hq, hkv, dh, dt, packed, far=T < 100)
    got = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, eps=1e-5, rope_base=1e4, rot_dim=rot)
    cos, sin = ops_ref.rotation(pos, rot, 1e4)
    fp = 32 * U if dt == torch.float32 else 2.0 ** -19
    for i, (x, w, dy, name) in enumerate(((q, wq, dq, "dq"), (k, wk, dk, "dk"))):
        dx, dw, size, dw_size = ops_ref.norm_rope_bwd(x, w, cos, sin, float(np.float32(1e-5)), dy)
        _close(got[i], dx, (torch.finfo(dt).eps / 2) * dx.abs() * (1 + 2.0 ** -7) + fp * size + 1e-37, name)
        _close(got[2 + i], dw, (64 * U + fp) * dw_size + 1e-37, name + "_weight")
    again = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, eps=1e-5, rope_base=1e4, rot_dim=rot)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "sums in a fixed order"


def test_backward_against_differences(api):
    # fp32: d/dh of sum(y dy) along a direction e; the forward's values are off by 16 u of
    # their size each, so a central difference over h is off by that sum / h, plus h^2
    T, hq, hkv, dh, rot = 3, 2, 1, 32, 16
    q, k, wq, wk, pos, dq, dk = _inputs(4, T, hq, hkv, dh, torch.float32, False)
    got = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, eps=1e-6, rot_dim=rot)

    def f(q, k, wq, wk):
        a, b = api.qk_norm_rope(q, k, wq, wk, pos, eps=1e-6, rot_dim=rot)
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())
    size = float(dq.abs().sum() * 4 + dk.abs().sum() * 2)
    h = 2.0 ** -7
    for i, x in enumerate((q, k, wq, wk)):
        g = torch.Generator().manual_seed(i)
        e = torch.randn(x.shape, generator=g).cuda()
        args = [q, k, wq, wk]
        up, dn = list(args), list(args)
        up[i], dn[i] = x + h * e, x - h * e
        num = (f(*up) - f(*dn)) / (2 * h)
        ana = float((got[i].double() * e.double()).sum())
        assert abs(num - ana) <= 17 * U * size / h + 8 * h * h * size, (i, num, ana)


def test_in_place_and_strided_outputs(api):
    T, hq, hkv, dh = 19, 4, 2, 128
    q, k, wq, wk, pos, dq, dk = _inputs(9, T, hq, hkv, dh, torch.bfloat16, True)
    want = api.qk_norm_rope(q, k, wq, wk, pos)
    buf = torch.full((T, hq + 2 * hkv, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    o = api.qk_norm_rope(q, k, wq, wk, pos, out=(buf[:, :hq], buf[:, hq:hq + hkv]))
    assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]) and (buf[:, hq + hkv:] == 7).all()
    gw = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk)
    gb = torch.zeros(T, hq + 2 * hkv, dh, dtype=torch.bfloat16, device="cuda")
    gi = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk,
                              grads=(gb[:, :hq], gb[:, hq:hq + hkv], torch.empty_like(wq), torch.empty_like(wk)))
    assert all(torch.equal(a, b) for a, b in zip(gw, gi)) and (gb[:, hq + hkv:] == 0).all()
    qc, kc = dq.clone(), dk.clone()   # dq over its own upstream gradient
    gi = api.qk_norm_rope_bwd(q, k, wq, wk, pos, qc, kc, grads=(qc, kc, torch.empty_like(wq), torch.empty_like(wk)))
    assert all(torch.equal(a, b) for a, b in zip(gw, gi))
    api.qk_norm_rope(q, k, wq, wk, pos, out=(q, k))   # in place, in the packed buffer
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_zero_rows_special_values_and_no_tokens(api):
    q = torch.zeros(2, 1, 64, device="cuda")
    q[1] = float("inf")
    w = torch.ones(64, device="cuda")
    pos = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    a, b = api.qk_norm_rope(q, q.clone(), w, w, pos)
    assert (a[0] == 0).all() and torch.isnan(a[1]).any()
    e = q[:0]
    a, b = api.qk_norm_rope(e, e, w, w, pos[:0])
    assert a.shape == (0, 1, 64)
    g = api.qk_norm_rope_bwd(e, e, w, w, pos[:0], e, e, grads=(e, e, torch.full_like(w, 9.0), torch.full_like(w, 9.0)))
    assert (g[2] == 0).all() and (g[3] == 0).all()


def test_no_rotation_at_position_zero(api):
    # rotation by zero is exact: the rows of a projection at position 0 are not rotated
    q, k, wq, wk, pos, _, _ = _inputs(3, 11, 4, 2, 128, torch.bfloat16, False)
    a = api.qk_norm_rope(q, k, wq, wk, torch.zeros_like(pos))
    b = api.qk_norm_rope(q, k, wq, wk, pos, rot_dim=0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_stream_and_graph(api):
    q, k, wq, wk, pos, dq, dk = _inputs(12, 40, 4, 2, 128, torch.bfloat16, False)
    want = api.qk_norm_rope(q, k, wq, wk, pos) + api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = api.qk_norm_rope(q, k, wq, wk, pos, stream=s) + api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = api.qk_norm_rope(q, k, wq, wk, pos) + api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk)
    q.mul_(2).add_(0.5)
    graph.replay()
    want = api.qk_norm_rope(q, k, wq, wk, pos) + api.qk_norm_rope_bwd(q, k, wq, wk, pos, dq, dk)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))
