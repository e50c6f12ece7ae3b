"""CPU side of the q/k norm with rotation, the quantised cache and the attention of
drafted tokens: their 64-bit references pinned by differences and by hand, the tree
mask helper, and every refusal of the C ABI and of the binding."""
import ctypes
import math

import pytest
import torch

import ops_ref
from learned_token_pruning_gemm_b200 import _lib, api, build
from learned_token_pruning_gemm_b200._lib import TokenGateError

INVALID, UNSUP, MIS, WS = 1, 2, 3, 4
F32, BF16, I8, E4M3 = 0, 1, 2, 3
P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10004)   # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def raises(match, fn, *a, **kw):
    with pytest.raises(TokenGateError, match=match):
        fn(*a, **kw)


# ---- references ----

def test_reference_gradient_matches_differences():
    g = torch.Generator().manual_seed(1)
    T, H, dh, rot = 3, 2, 16, 8
    x = torch.randn(T, H, dh, generator=g, dtype=torch.float64)
    w = 0.5 + torch.rand(dh, generator=g, dtype=torch.float64)
    dy = torch.randn(T, H, dh, generator=g, dtype=torch.float64)
    cos, sin = ops_ref.rotation(torch.tensor([0, 5, 70000]), rot, 1e4)
    dx, dw, _, _ = ops_ref.norm_rope_bwd(x, w, cos, sin, 1e-6, dy)
    f = lambda x, w: float((ops_ref.norm_rope(x, w, cos, sin, 1e-6) * dy).sum())
    h = 1e-6   # central differences: h^2 from the third derivative, 2^-53 * |f| / h from rounding
    for t, hd, d in ((0, 0, 0), (1, 1, 5), (2, 0, 3), (2, 1, 15)):
        e = torch.zeros_like(x)
        e[t, hd, d] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx[t, hd, d])) < 1e-7
    for d in (0, 7, 15):
        e = torch.zeros_like(w)
        e[d] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[d])) < 1e-7


def test_reference_codes_by_hand():
    x = torch.tensor([[127.0, 0.5, 1.5, -2.5, 0.0, 126.5, -127.0, 1.0]]).to(torch.bfloat16)
    x[0, 5] = 63.5
    v, s = ops_ref.quantise(x, torch.int8)
    assert s.item() == 1.0 and v[0].tolist() == [127, 0, 2, -2, 0, 64, -127, 1]   # ties to even
    x = torch.tensor([[448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -0.25, 23.0, 1.0625]]).to(torch.bfloat16)
    v, s = ops_ref.quantise(x, torch.float8_e4m3fn)
    assert s.item() == 1.0
    assert v[0].tolist() == [448.0, 16.0, 20.0, 0.0, 2.0 ** -8, -0.25, 24.0, 1.0]
    x = torch.tensor([[float("inf"), 1.0], [0.0, 0.0], [1e-30, 0.0]]).to(torch.bfloat16)
    v, s = ops_ref.quantise(x, torch.int8)
    assert math.isnan(s[0].item()) and s[1:].tolist() == [0.0, 0.0] and (v == 0).all()


def test_tree_mask():
    m = api.tree_mask([[-1, 0, 0, 2, -1], [-1]])
    assert m.tolist() == [[1, 3, 5, 13, 16], [1, 0, 0, 0, 0]]
    chain = api.tree_mask([list(range(-1, 63))])
    assert chain[0, 63].item() == -1 and chain[0, 62].item() == 2 ** 63 - 1
    assert api.tree_mask([]).shape == (0, 0) and api.tree_mask([[]]).shape == (1, 0)
    raises("parents\\[0\\]\\[1\\]", api.tree_mask, [[-1, 1]])
    raises("must be in", api.tree_mask, [[-2]])
    raises("at most 64", api.tree_mask, [[-1] * 65])


# ---- refusals of the C ABI ----

def test_norm_rope_refusals(lib):
    def fwd(q=FAKE, qs=2048, k=FAKE, ks=1024, dt=BF16, T=10, hq=16, hkv=8, dh=128, rot=128, wq=FAKE,
            eps=1e-6, base=1e6, pos=FAKE, qo=FAKE, qos=2048, ko=FAKE, kos=1024):
        return lib.tg_qk_norm_rope(q, qs, k, ks, dt, T, hq, hkv, dh, rot, wq, FAKE, eps, base, pos, qo,
                                   qos, ko, kos, None)
    assert fwd(T=0, q=None) == 0
    for kw in (dict(q=None), dict(k=None), dict(wq=None), dict(pos=None), dict(qo=None), dict(ko=None),
               dict(T=-1), dict(hq=0), dict(rot=136), dict(rot=-8), dict(eps=-1.0),
               dict(eps=float("nan")), dict(base=1.0), dict(base=float("inf")), dict(qs=2047),
               dict(ks=1016), dict(qos=8), dict(kos=0)):
        assert fwd(**kw) == INVALID, kw
    for kw in (dict(dt=I8), dict(dt=7), dict(dh=100, rot=96), dict(rot=12),
               dict(dh=264, rot=8, qs=16 * 264, ks=8 * 264, qos=16 * 264, kos=8 * 264)):
        assert fwd(**kw) == UNSUP, kw
    for kw in (dict(q=ODD), dict(ko=ODD), dict(qs=2052), dict(kos=1026), dict(dt=F32, qs=2050)):
        assert fwd(**kw) == MIS, kw
    size = lib.tg_qk_norm_rope_bwd_workspace_size
    need = size(10, 16, 8, 128)
    assert need > 0 and size(0, 16, 8, 128) == 0 and size(10, 16, 8, 300) == 0

    def bwd(q=FAKE, dq=FAKE, dqs=2048, dwq=FAKE, ws=FAKE, nb=need, T=10, gq=FAKE, gqs=2048):
        return lib.tg_qk_norm_rope_bwd(q, 2048, FAKE, 1024, gq, gqs, FAKE, 1024, BF16, T, 16, 8, 128, 128,
                                       FAKE, FAKE, 1e-6, 1e6, FAKE, dq, dqs, FAKE, 1024, dwq, FAKE, ws, nb,
                                       None)
    for kw in (dict(q=None), dict(dq=None), dict(dwq=None), dict(gq=None), dict(dqs=2040),
               dict(gqs=1), dict(T=-1), dict(T=0, dwq=None)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(ws=None) == WS and bwd(nb=need - 1) == WS
    assert bwd(ws=ODD) == MIS and bwd(dq=ODD) == MIS and bwd(gqs=2050) == MIS


def test_quant_cache_refusals(lib):
    def app(k=FAKE, n_src=5, idx=None, n=5, cu=FAKE, start=None, B=2, cap=10, hkv=8, dh=128, dt=I8,
            kc=FAKE, ks=FAKE, sc=FAKE, ln=P(0x20000)):
        return lib.tg_quant_cache_append(k, FAKE, FAKE, n_src, idx, n, cu, start, B, cap, hkv, dh, dt, kc,
                                         FAKE, ks, FAKE, sc, ln, None)
    assert app(B=0, cu=None, ln=None) == 0
    for kw in (dict(k=None), dict(cu=None), dict(kc=None), dict(ks=None), dict(sc=None), dict(ln=None),
               dict(n=4), dict(n=-1), dict(n_src=-1), dict(B=-1), dict(cap=0), dict(hkv=0),
               dict(start=P(0x20004)), dict(start=P(0x1fffc))):
        assert app(**kw) == INVALID, kw
    for kw in (dict(dh=96), dict(dt=BF16), dict(dt=F32), dict(B=70000)):
        assert app(**kw) == UNSUP, kw
    for kw in (dict(k=ODD), dict(kc=ODD)):
        assert app(**kw) == MIS, kw

    def rd(kc=FAKE, ks=FAKE, ln=FAKE, cu=FAKE, n=5, B=2, cap=10, dh=128, dt=E4M3, odt=BF16, k=FAKE, s=FAKE):
        return lib.tg_quant_cache_read(kc, FAKE, ks, FAKE, FAKE, ln, None, cu, n, B, cap, 8, dh, dt, odt, k,
                                       FAKE, s, None)
    assert rd(n=0, k=None, s=None) == 0 and rd(B=0) == 0
    for kw in (dict(kc=None), dict(ks=None), dict(ln=None), dict(cu=None), dict(k=None), dict(s=None),
               dict(n=-1), dict(cap=0)):
        assert rd(**kw) == INVALID, kw
    for kw in (dict(dh=32), dict(dt=BF16), dict(odt=I8)):
        assert rd(**kw) == UNSUP, kw
    assert rd(k=ODD) == MIS and rd(kc=ODD) == MIS


def test_tree_attention_refusals(lib):
    need = lib.tg_tree_attention_workspace_size(2, 8, 100, 16, 8, 128)
    assert need > 0 and lib.tg_tree_attention_workspace_size(0, 8, 100, 16, 8, 128) == 0

    def run(q=FAKE, mask=FAKE, B=2, T=8, kc=FAKE, dt=BF16, ks=None, vs=None, ln=FAKE, cap=100, ml=100,
            hq=16, hkv=8, dh=128, gain=FAKE, out=FAKE, ws=FAKE, nb=need, dl=None):
        return lib.tg_tree_attention(q, FAKE, FAKE, FAKE, mask, dl, B, T, kc, FAKE, dt, ks, vs, FAKE, ln, cap,
                                     ml, hq, hkv, dh, gain, FAKE, out, ws, nb, None)
    assert run(B=0, q=None) == 0 and run(T=0, q=None) == 0
    for kw in (dict(q=None), dict(mask=None), dict(kc=None), dict(ln=None), dict(gain=None),
               dict(out=None), dict(B=-1), dict(T=-1), dict(cap=0), dict(ml=101), dict(ml=-1),
               dict(hq=15), dict(hkv=0), dict(ks=FAKE), dict(vs=FAKE), dict(dt=I8),
               dict(dt=E4M3, ks=FAKE)):
        assert run(**kw) == INVALID, kw
    for kw in (dict(dt=F32), dict(dt=9), dict(dh=96), dict(T=65), dict(hq=8 * 129), dict(B=1025),
               dict(B=1024, cap=1 << 22, ml=100)):
        assert run(**kw) == UNSUP, kw
    for kw in (dict(q=ODD), dict(kc=ODD), dict(out=ODD), dict(ws=ODD)):
        assert run(**kw) == MIS, kw
    assert run(ws=None) == WS and run(nb=need - 1) == WS


# ---- refusals of the binding, before any call ----

def test_binding_norm_rope_checks():
    T, hq, hkv, dh = 5, 4, 2, 64
    q, k = torch.zeros(T, hq, dh), torch.zeros(T, hkv, dh)
    w, pos = torch.zeros(dh), torch.zeros(T, dtype=torch.int32)
    f = api.qk_norm_rope
    raises("q_weight must have shape", f, q, k, w[:-1], w, pos)
    raises("k_weight must be", f, q, k, w, w.double(), pos)
    raises("pos must be", f, q, k, w, w, pos.long())
    raises("pos must have shape", f, q, k, w, w, pos[:-1])
    raises("unsupported dtype", f, q.half(), k.half(), w, w, pos)
    raises("k must be", f, q, k.bfloat16(), w, w, pos)
    raises("dense heads", f, q.transpose(0, 1).contiguous().transpose(0, 1), k, w, w, pos)
    raises("q_out must have shape", f, q, k, w, w, pos, out=(q[:, :1], k))
    raises("CUDA tensor", f, q, k, w, w, pos)
    g = api.qk_norm_rope_bwd
    raises("dq_out must have shape", g, q, k, w, w, pos, q[:-1], k)
    raises("dk_out must be", g, q, k, w, w, pos, q, k.bfloat16())
    raises("dq_weight must have shape", g, q, k, w, w, pos, q, k, grads=(q, k, w[:-1], w))


def test_binding_quant_cache_checks():
    B, cap, hkv, dh, R = 2, 10, 2, 64, 5
    kc = torch.zeros(B, cap, hkv, dh, dtype=torch.int8)
    sc, ss = torch.zeros(B, cap, hkv), torch.zeros(B, cap)
    ln, cu = torch.zeros(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    x, s = torch.zeros(R, hkv, dh, dtype=torch.bfloat16), torch.zeros(R)
    f = api.quant_cache_append
    raises("int8 or float8", f, x, x, s, cu, kc.bfloat16(), kc, sc, sc, ss, ln)
    raises("v_cache must", f, x, x, s, cu, kc, kc.view(torch.float8_e4m3fn), sc, sc, ss, ln)
    raises("v_scale must have shape", f, x, x, s, cu, kc, kc, sc, sc[:1], ss, ln)
    raises("s_cache must have shape", f, x, x, s, cu, kc, kc, sc, sc, ss[:, 1:], ln)
    raises("k_new must be", f, x.float(), x, s, cu, kc, kc, sc, sc, ss, ln)
    raises("v_new must have shape", f, x, x[1:], s, cu, kc, kc, sc, sc, ss, ln)
    raises("cu_new must have shape", f, x, x, s, cu[1:], kc, kc, sc, sc, ss, ln)
    raises("src_idx must be", f, x, x, s, cu, kc, kc, sc, sc, ss, ln, src_idx=torch.zeros(3))
    raises("start must have shape", f, x, x, s, cu, kc, kc, sc, sc, ss, ln, start=cu)
    raises("CUDA tensor", f, x, x, s, cu, kc, kc, sc, sc, ss, ln)
    r = api.quant_cache_read
    raises("cu_rows must have shape", r, kc, kc, sc, sc, ss, ln, ln, 5)
    raises("unsupported dtype", r, kc, kc, sc, sc, ss, ln, cu, 5, dtype=torch.float16)
    raises("k must have shape", r, kc, kc, sc, sc, ss, ln, cu, 5, out=(x[1:], x, s))


def test_binding_tree_checks():
    B, T, hq, hkv, dh, cap = 2, 3, 4, 2, 64, 10
    bf = dict(dtype=torch.bfloat16)
    q, d = torch.zeros(B, T, hq, dh, **bf), torch.zeros(B, T, hkv, dh, **bf)
    sd, m = torch.zeros(B, T), torch.zeros(B, T, dtype=torch.int64)
    kc, sc = torch.zeros(B, cap, hkv, dh, **bf), torch.zeros(B, cap)
    ln, g = torch.zeros(B, dtype=torch.int32), torch.zeros(hq)
    f = lambda q=q, kd=d, vd=d, sd=sd, m=m, kc=kc, vc=kc, sc=sc, ln=ln, g=g, t=g, **kw: \
        api.tree_attention(q, kd, vd, sd, m, kc, vc, sc, ln, g, t, cap, **kw)
    raises("q \\[B,T,Hq,dh\\]", f, q=q[0])
    raises("k_draft must have shape", f, kd=d[:, 1:])
    raises("v_draft must be", f, vd=d.float())
    raises("tree_mask must be", f, m=m.int())
    raises("s_draft must have shape", f, sd=sd[:, 1:])
    raises("k_cache must have shape", f, kc=kc[:1])
    raises("v_cache must be", f, vc=kc.float())
    raises("cache_len must be", f, ln=ln.long())
    raises("gain must have shape", f, g=g[1:])
    raises("tau must have shape", f, t=g[1:])
    raises("needs k_scale and v_scale", f, kc=kc.to(torch.int8), vc=kc.to(torch.int8))
    raises("bf16 without scales", f, k_scale=sc, v_scale=sc)
    raises("bf16 without scales", f, kc=kc.float(), vc=kc.float())
    raises("draft_len must be", f, draft_len=ln.long())
    raises("out must be", f, out=q.float())
    raises("CUDA tensor", f)
