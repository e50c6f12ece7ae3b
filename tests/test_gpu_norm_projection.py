"""GPU test of a layer that normalises q and k per head, as include/tg.h describes it: the
projection without rotation (tg_qkv_rope at position 0 for every row), tg_qk_norm_rope at
the kept tokens' positions, then the gated attention over the result, or the quantised
cache and a single token over it. Every stage against its 64-bit form on its own inputs."""
import math

import pytest
import torch

import ops_ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8          # half a step of bf16
EPS, BASE = 1e-6, 1e6


@pytest.fixture(scope="module")
def api():
    from learned_token_pruning_gemm_b200 import api, build
    build.build()
    api.device_status(reset=True)
    return api


def _close(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


@pytest.mark.parametrize("lens,hq,hkv", [([130, 1, 257], 4, 2), ([64], 16, 8)])
def test_normed_layer(api, lens, hq, hkv):
    g = torch.Generator().manual_seed(sum(lens))
    d, dh, K = 256, 128, sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    xc, w = rnd(K, d).to(BF), (rnd((hq + 2 * hkv) * dh, d) / 16).to(BF)
    wq, wk, s = 1 + 0.1 * rnd(dh), 1 + 0.1 * rnd(dh), rnd(K)
    gain, tau = torch.rand(hq, generator=g).cuda(), (0.8 + 0.7 * torch.rand(hq, generator=g)).cuda()
    pos = torch.cat([torch.sort(torch.randperm(5000, generator=g)[:n])[0] for n in lens]).to(torch.int32).cuda()

    # the projection: sums of d fp32 products, stored once; position 0 is the identity rotation
    q0, k0, v = api.qkv_rope(xc, w, hq, hkv, torch.zeros_like(pos))
    z = xc.double() @ w.double().T
    size = xc.double().abs() @ w.double().abs().T
    for got, r in ((q0, slice(0, hq * dh)), (k0, slice(hq * dh, (hq + hkv) * dh)), (v, slice((hq + hkv) * dh, None))):
        want = z[:, r].reshape(K, -1, dh)
        _close(got, want, HALF * want.abs() * (1 + HALF) + d * 2.0 ** -24 * size[:, r].reshape(K, -1, dh))

    # norm and rotation, over the projection's own outputs
    q, k = api.qk_norm_rope(q0, k0, wq, wk, pos, EPS, BASE, out=(q0.clone(), k0.clone()))
    cos, sin = ops_ref.rotation(pos, dh, BASE)
    for got, x, wx in ((q, q0, wq), (k, k0, wk)):
        n = x.double() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + EPS) * wx.double()
        want = ops_ref.rotate(n, cos, sin)
        _close(got, want, HALF * want.abs() * (1 + 2 * HALF) + 2.0 ** -20 * ops_ref.pair_size(n, cos) + 1e-37)

    # the gated attention over them: weights and outputs are rounded to bf16, the exponential is off
    # by 2^-13 at most, logits by less than 2^-12
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    out = api.gated_attention(q, k, v, s, gain, tau, cu, max(lens))
    off = 0
    for n in lens:
        r = slice(off, off + n)
        kk, vv = (t[r].double().repeat_interleave(hq // hkv, 1) for t in (k, v))
        z = torch.einsum("thd,nhd->htn", q[r].double(), kk) / (math.sqrt(dh) * tau.double()[:, None, None])
        z = z + gain.double()[:, None, None] * s[r].double()
        p = z.masked_fill(torch.ones(n, n, dtype=torch.bool).cuda().triu(1), float("-inf")).softmax(-1)
        o = torch.einsum("htn,nhd->thd", p, vv)
        # sum p |v - o| <= sum p |v| + |o|
        spread = torch.einsum("htn,nhd->thd", p, vv.abs()) + o.abs()
        _close(out[r], o, HALF * o.abs() * (1 + 2 * HALF) + (HALF * (1 + 2 * HALF) + 2.0 ** -12 + 2.0 ** -13) * spread + 1e-6)
        off += n

    # the rows enter a quantised cache, and a single token of the same layer attends over it
    B, cap = len(lens), max(lens)
    z8 = lambda *sh, dt=torch.float32: torch.zeros(*sh, dtype=dt).cuda()
    kc, vc = z8(B, cap, hkv, dh, dt=torch.int8), z8(B, cap, hkv, dh, dt=torch.int8)
    ks, vs, sc, ln = z8(B, cap, hkv), z8(B, cap, hkv), z8(B, cap), z8(B, dt=torch.int32)
    api.quant_cache_append(k, v, s, cu, kc, vc, ks, vs, sc, ln)
    xt = rnd(B, d).to(BF)
    qt, kt, vt = api.qkv_rope(xt, w, hq, hkv, z8(B, dt=torch.int32))
    qt, kt = api.qk_norm_rope(qt, kt, wq, wk, torch.full((B,), 5000, dtype=torch.int32).cuda(), EPS, BASE)
    st, one = rnd(B, 1), torch.ones(B, 1, dtype=torch.int64).cuda()
    o = api.tree_attention(qt[:, None], kt[:, None], vt[:, None], st, one, kc, vc, sc, ln, gain, tau, cap, k_scale=ks,
                           v_scale=vs)
    want, spread = ops_ref.tree_attention(qt[:, None], kt[:, None], vt[:, None], st, one.cpu(), kc.double() * ks.double()[..., None],
                                          vc.double() * vs.double()[..., None], sc, lens, [1] * B, gain.cpu(), tau.cpu())
    _close(o, want, HALF * want.abs() * (1 + HALF) + HALF * spread + 2.0 ** -11 * want.abs() + 1e-6)
    assert api.device_status(reset=True) == 0
