"""The q/k norm with rotation, the quantised cache and the attention of drafted tokens
together, as generation and training run them: what one call leaves on the device is what
the next one reads, and nothing goes through the host in between."""
import pytest
import torch

import ops_ref

pytestmark = pytest.mark.gpu
BF, I8, E4 = torch.bfloat16, torch.int8, torch.float8_e4m3fn
HQ, HKV, EPS, BASE = 16, 8, 1e-6, 1e6


@pytest.fixture(scope="module")
def api():
    from learned_token_pruning_gemm_b200 import api, build
    build.build()
    api.device_status(reset=True)
    return api


@pytest.fixture(autouse=True)
def _status(api):
    yield
    assert api.device_status(reset=True) == 0, "a kernel recorded a device-side error"


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _cu(counts):
    return _i32([sum(counts[:i]) for i in range(len(counts) + 1)])


class Serving:
    """Prompts of which some rows are kept, then a tree of drafted tokens of which some are
    accepted, then single tokens."""

    def __init__(self, api, fmt, dh, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.api, self.fmt, self.dh = api, fmt, dh
        rnd = lambda *s: torch.randn(*s, generator=g)
        self.prompts, self.cap, self.T = [150, 9, 300], 260, 5
        B, R, T = len(self.prompts), sum(self.prompts), self.T
        width = (HQ + 2 * HKV) * dh
        packed = lambda n: rnd(n, width).to(BF).cuda()
        self.x, self.x_draft, self.x_one = packed(R), packed(B * T), packed(B)
        self.wq, self.wk = (1 + 0.1 * rnd(dh)).cuda(), (1 + 0.1 * rnd(dh)).cuda()
        self.gain, self.tau = torch.rand(HQ, generator=g).cuda(), (0.8 + 0.7 * torch.rand(HQ, generator=g)).cuda()
        self.s, self.s_draft, self.s_one = rnd(R).cuda(), rnd(B, T).cuda(), rnd(B, 1).cuda()
        keep, off = [], 0
        for n in self.prompts:   # every third row goes
            keep.append([off + i for i in range(n) if i % 3 != 1])
            off += n
        self.kept = [len(k) for k in keep]
        self.idx = _i32([i for k in keep for i in k])
        self.pos = _i32([i for n in self.prompts for i in range(n)])
        parents = [[-1, 0, 0, 1, -1]] * B
        self.mask = api.tree_mask(parents).cuda()
        depth = [0, 1, 1, 2, 0]
        self.pos_draft = _i32([n + d for n in self.prompts for d in depth])
        self.accept = [[0, 2], [4], [0, 1, 3]]           # a path of each tree
        self.idx_accept = _i32([b * T + t for b, a in enumerate(self.accept) for t in a])
        self.pos_one = _i32([n + len(a) for n, a in zip(self.prompts, self.accept)])
        self.one = torch.ones(B, 1, dtype=torch.int64).cuda()
        self.cu_kept, self.cu_accept = _cu(self.kept), _cu([len(a) for a in self.accept])
        self.total = sum(self.kept) + sum(len(a) for a in self.accept)
        self.cu_all = _cu([k + len(a) for k, a in zip(self.kept, self.accept)])
        z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt).cuda()
        self.c = dict(kc=z(B, self.cap, HKV, dh, dt=fmt), vc=z(B, self.cap, HKV, dh, dt=fmt),
                      ks=z(B, self.cap, HKV), vs=z(B, self.cap, HKV), sc=z(B, self.cap), len=z(B, dt=torch.int32))

    def heads(self, x, pos):
        n = x.shape[0]
        q, k, v = x.split([HQ * self.dh, HKV * self.dh, HKV * self.dh], 1)
        q, k = self.api.qk_norm_rope(q.view(n, HQ, self.dh), k.view(n, HKV, self.dh), self.wq, self.wk, pos, EPS, BASE)
        return q, k, v.reshape(n, HKV, self.dh).contiguous()

    def append(self, k, v, s, cu, idx):
        c = self.c
        self.api.quant_cache_append(k, v, s, cu, c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], c["len"], src_idx=idx)

    def attend(self, q, k, v, s, mask):
        c, B = self.c, len(self.prompts)
        v4 = lambda t: t.view(B, -1, t.shape[1], self.dh)
        return self.api.tree_attention(v4(q), v4(k), v4(v), s, mask, c["kc"], c["vc"], c["sc"], c["len"], self.gain,
                                       self.tau, self.cap, k_scale=c["ks"], v_scale=c["vs"])

    def __call__(self):
        self.c["len"].zero_()
        self.p = self.heads(self.x, self.pos)
        self.append(self.p[1], self.p[2], self.s, self.cu_kept, self.idx)
        self.d = self.heads(self.x_draft, self.pos_draft)
        self.out = self.attend(*self.d, self.s_draft, self.mask)
        self.append(self.d[1], self.d[2], self.s_draft.view(-1), self.cu_accept, self.idx_accept)
        self.o = self.heads(self.x_one, self.pos_one)
        self.out_one = self.attend(*self.o, self.s_one, self.one)
        self.read = self.api.quant_cache_read(self.c["kc"], self.c["vc"], self.c["ks"], self.c["vs"], self.c["sc"],
                                              self.c["len"], self.cu_all, self.total)
        return self.out, self.out_one, *self.read


def _check_attention(S, got, heads, s, mask, lens):
    """Against the 64-bit form on what the cache holds (rows are only added behind), at
    twice the tolerance of a weight and an output rounded to bf16."""
    B, c = len(lens), S.c
    v4 = lambda t: t.view(B, -1, t.shape[1], S.dh)
    k, v = (c[n + "c"].double() * c[n + "s"].double()[..., None] for n in "kv")
    T = got.shape[1]
    want, spread = ops_ref.tree_attention(*(v4(t) for t in heads), s, mask.cpu(), k, v, c["sc"], lens, [T] * B,
                                          S.gain.cpu(), S.tau.cpu())
    assert ((got.double() - want).abs() <= 2.0 ** -7 * (want.abs() + spread) + 1e-6).all()


@pytest.mark.parametrize("fmt,dh", [(I8, 128), (E4, 128), (I8, 64), (E4, 64)])
def test_generation_on_a_quantised_cache(api, fmt, dh):
    S = Serving(api, fmt, dh)
    S()
    B = len(S.prompts)
    lens = [k + len(a) for k, a in zip(S.kept, S.accept)]
    assert S.c["len"].tolist() == lens
    # what was stored: the rotated rows of kept and accepted tokens, quantised as defined
    cos, sin = ops_ref.rotation(S.pos, dh, BASE)
    x = S.x[:, HQ * dh:(HQ + HKV) * dh].reshape(-1, HKV, dh)
    size = ops_ref.pair_size(ops_ref.norm_rope(x, S.wk, cos, sin, EPS), cos)
    assert ((S.p[1].double() - ops_ref.norm_rope(x, S.wk, cos, sin, EPS)).abs()
            <= 2.0 ** -8 * (1 + 2.0 ** -7) * size + 2.0 ** -18 * size).all()
    r = a = 0
    for b in range(B):
        n, m = S.kept[b], len(S.accept[b])
        for i, nm in ((1, "k"), (2, "v")):
            rows = torch.cat([S.p[i][S.idx[r:r + n].long()], S.d[i][S.idx_accept[a:a + m].long()]])
            code, scale = ops_ref.quantise(rows, fmt)
            assert torch.equal(S.c[nm + "c"][b, :n + m].double(), code)
            assert torch.equal(S.c[nm + "s"][b, :n + m], scale)
            packed = S.read[i - 1][r + a:r + a + n + m]
            assert torch.equal(packed, (code.float() * scale[..., None]).to(BF))
        s = torch.cat([S.s[S.idx[r:r + n].long()], S.s_draft.view(-1)[S.idx_accept[a:a + m].long()]])
        assert torch.equal(S.c["sc"][b, :n + m], s) and torch.equal(S.read[2][r + a:r + a + n + m], s)
        r, a = r + n, a + m
    _check_attention(S, S.out, S.d, S.s_draft, S.mask, S.kept)
    _check_attention(S, S.out_one, S.o, S.s_one, S.one, lens)


def test_generation_captured_and_replayed(api):
    # the whole run as one graph, on its own stream, replayed over other inputs
    S, W = Serving(api, E4, 128, seed=2), Serving(api, E4, 128, seed=3)
    want = [t.clone() for t in W()]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        S()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = S()
    for n in ("x", "x_draft", "x_one", "wq", "wk", "gain", "tau", "s", "s_draft", "s_one"):
        getattr(S, n).copy_(getattr(W, n))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_training_step_of_normed_attention(api):
    # norm and rotation, gated attention, and both backward passes, in fp32, against the
    # derivative of the whole formula in 64 bits
    g = torch.Generator().manual_seed(4)
    lens, hq, hkv, dh, rot = [37, 1, 64], 4, 2, 64, 32
    K = sum(lens)
    rnd = lambda *s: torch.randn(*s, generator=g).cuda()
    q, k, v, dout = rnd(K, hq, dh), rnd(K, hkv, dh), rnd(K, hkv, dh), rnd(K, hq, dh)
    wq, wk = 1 + 0.1 * rnd(dh), 1 + 0.1 * rnd(dh)
    s, gain, tau = rnd(K), torch.rand(hq, generator=g).cuda(), (0.8 + torch.rand(hq, generator=g)).cuda()
    pos, cu = _i32([3 * i for n in lens for i in range(n)]), _cu(lens)
    qr, kr = api.qk_norm_rope(q, k, wq, wk, pos, EPS, BASE, rot)
    lse = torch.empty(hq, K).cuda()
    out = api.gated_attention(qr, kr, v, s, gain, tau, cu, max(lens), lse=lse)
    dqr, dkr, dv, ds, _, _ = api.gated_attention_bwd(qr, kr, v, out, dout, lse, s, gain, tau, cu, max(lens))
    dq, dk, dwq, dwk = api.qk_norm_rope_bwd(q, k, wq, wk, pos, dqr, dkr, EPS, BASE, rot)

    leaves = [t.double().requires_grad_() for t in (q, k, v, s, wq, wk)]
    q6, k6, v6, s6, wq6, wk6 = leaves
    cos, sin = ops_ref.rotation(pos, rot, BASE)
    norm = lambda x, w: ops_ref.rotate(x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w, cos, sin)
    qn, kn, off, total = norm(q6, wq6), norm(k6, wk6), 0, 0.0
    for n in lens:
        r = slice(off, off + n)
        kk, vv = (t[r].repeat_interleave(hq // hkv, 1) for t in (kn, v6))
        z = torch.einsum("thd,nhd->htn", qn[r], kk) / (dh ** 0.5 * tau.double()[:, None, None])
        z = z + gain.double()[:, None, None] * s6[r]
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool).cuda().triu(1), float("-inf"))
        o = torch.einsum("htn,nhd->thd", z.softmax(-1), vv)
        # four fp32 stages with sums of at most 64 terms (2^-24 each, fast exponentials 2^-22)
        assert ((out[r].double() - o).abs() <= 2.0 ** -14 * vv.abs().max()).all()
        total = total + (o * dout[r].double()).sum()
        off += n
    want = torch.autograd.grad(total, leaves)
    for name, a, b in zip(("dq", "dk", "dv", "ds", "dwq", "dwk"), (dq, dk, dv, ds, dwq, dwk), want):
        # as above, and a gradient's terms may exceed it: by less than four times its largest
        assert ((a.double() - b).abs() <= 2.0 ** -12 * b.abs().max()).all(), name


@pytest.mark.parametrize("fmt", [I8, BF])
@pytest.mark.parametrize("T,dh", [(1, 128), (12, 128), (3, 64)])
def test_offsets_behind_32_bits(api, fmt, T, dh):
    # the last sequence of a cache of more than 2^31 elements, as it is in a cache of its own
    from test_gpu_tree_attn import check, make, reference, run
    cap, n, hkv = 60000, 1500, HKV
    B = 2 ** 31 // (cap * hkv * dh) + 2
    small = make(41, 1, T, cap, [n], HQ, hkv, dh, fmt, garbage=False)
    st = {}
    for name, t in small.items():
        st[name] = t if t is None or name in ("gain", "tau") else torch.empty((B,) + t.shape[1:], dtype=t.dtype,
                                                                              device=t.device)
        if st[name] is not None and st[name] is not t:
            st[name][-1] = t[0]
            if name in ("len", "dl"):
                st[name][:-1] = 0
    assert st["kc"].numel() > 2 ** 31
    out = torch.full_like(st["q"], 9.0)
    if fmt == BF:
        check(run(api, st, out=out)[-1:], reference(small))
        return
    # rows are appended behind those there, attended over, and read back
    g = torch.Generator().manual_seed(42)
    rows = 77
    k, v, s = (torch.randn(rows, hkv, dh, generator=g).to(BF).cuda(), torch.randn(rows, hkv, dh, generator=g).to(BF).cuda(),
               torch.randn(rows, generator=g).cuda())
    for c in (st, small):
        m = c["len"].numel()
        c["start"] = c["len"].clone()
        api.quant_cache_append(k, v, s, _i32([0] * m + [rows]), c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], c["len"])
        c["read"] = api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], c["len"], _i32([0] * m + [rows]),
                                         rows, start=c["start"])
    assert int(st["len"][-1]) == n + rows and not st["len"][:-1].any()
    for a, b in zip(st["read"], small["read"]):
        assert torch.equal(a, b)
    for name in ("kc", "vc", "ks", "vs", "sc"):
        assert torch.equal(st[name][-1, :n + rows], small[name][0, :n + rows])
    check(run(api, st, out=out)[-1:], reference(small))
