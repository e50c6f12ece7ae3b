"""GPU tests of the quantised cache: codes and scales are compared bit for bit with the
64-bit definition (ops_ref.quantise), rows given back with code * scale rounded once."""
import pytest
import torch

import ops_ref

pytestmark = pytest.mark.gpu
FMTS = [torch.int8, torch.float8_e4m3fn]


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


def _cu(counts):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32).cuda()


def _empty(B, cap, hkv, dh, fmt, seed=0):
    """A cache with something in every place, so that what a call leaves alone shows."""
    g = torch.Generator().manual_seed(seed)
    code = lambda: torch.randint(0, 120, (B, cap, hkv, dh), generator=g, dtype=torch.uint8).cuda().view(fmt)
    f = lambda *s: torch.rand(*s, generator=g).cuda()
    return dict(kc=code(), vc=code(), ks=f(B, cap, hkv), vs=f(B, cap, hkv), sc=f(B, cap))


def _rows(seed, R, hkv, dh):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, R, hkv, dh, generator=g) * torch.exp2(torch.randint(-6, 7, (2, R, hkv, 1), generator=g).float())
    x = x.to(torch.bfloat16)
    # few-bit rows: their quotients lie on borders between codes as often as not
    x[:, ::3] = (torch.round(x[:, ::3].float() * 8) / 8).to(torch.bfloat16)
    if R:
        x[0, 0, 0] = 0
        x[:, R // 2, 0, 1] = 448.0
    return x[0].cuda(), x[1].cuda(), torch.randn(R, generator=g).cuda()


def _append(api, c, ln, k, v, s, cu, **kw):
    api.quant_cache_append(k, v, s, cu, c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, **kw)


def _expect(c, k, v, s, counts, start, idx=None):
    """The cache as it should be, from its state before."""
    c = {n: t.clone() for n, t in c.items()}
    r = 0
    for b, n in enumerate(counts):
        for j in range(n):
            src = r if idx is None else int(idx[r])
            for name, x in (("k", k), ("v", v)):
                q, sc = ops_ref.quantise(x[src], c["kc"].dtype)
                c[name + "c"][b, start[b] + j] = q.to(torch.float32).to(c["kc"].dtype)
                c[name + "s"][b, start[b] + j] = sc
            c["sc"][b, start[b] + j] = s[src]
            r += 1
    return c


def _same(a, b):
    for n in a:
        if n in ("kc", "vc"):   # -0 and 0 stand for one value
            x, y = a[n].float(), b[n].float()
            assert torch.equal(x, y), (n, int((x != y).sum()))
        else:
            assert torch.equal(torch.nan_to_num(a[n], nan=-77.0), torch.nan_to_num(b[n], nan=-77.0)), n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts,cap,hkv,dh", [
    ([1], 1, 1, 128), ([5, 0, 3], 9, 8, 128), ([1, 1, 1, 1, 1], 4, 3, 64), ([0, 0], 5, 2, 64),
    ([40, 3, 0, 17] * 9, 64, 2, 128), ([700, 311], 800, 4, 64),
])
def test_append(api, fmt, counts, cap, hkv, dh):
    B, R = len(counts), sum(counts)
    start = [min(b % 3, cap - n) for b, n in enumerate(counts)]
    k, v, s = _rows(R, R, hkv, dh)
    c = _empty(B, cap, hkv, dh, fmt)
    want = _expect(c, k, v, s, counts, start)
    ln = torch.tensor(start, dtype=torch.int32).cuda()
    _append(api, c, ln, k, v, s, _cu(counts))
    assert ln.tolist() == [a + n for a, n in zip(start, counts)]
    _same(c, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_picks_rows_and_starts_anywhere(api, fmt):
    hkv, dh, cap, counts = 4, 128, 50, [2, 0, 4, 1]
    k, v, s = _rows(3, 30, hkv, dh)
    idx = torch.tensor([7, 8, 29, 0, 8, 8, 15], dtype=torch.int32).cuda()   # the same row twice
    start = [48, 3, 0, 20]
    c = _empty(4, cap, hkv, dh, fmt)
    want = _expect(c, k, v, s, counts, start, idx)
    ln = torch.full((4,), 33, dtype=torch.int32).cuda()
    _append(api, c, ln, k, v, s, _cu(counts), start=torch.tensor(start, dtype=torch.int32).cuda(), src_idx=idx)
    assert ln.tolist() == [50, 3, 4, 21]
    _same(c, want)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_values_to_the_code(api, fmt):
    # every bf16 magnitude against several row maxima: the code of the exact quotient
    bits = torch.arange(0x3000, 0x4700, dtype=torch.int32)
    vals = (bits << 16).view(torch.float32).to(torch.bfloat16)
    rows = []
    for top in (1.0, 1.75, 448.0, 127.0, 3.0, 100.5, 5.0, 0.4375):
        x = vals[vals.float() <= top].float()
        x = torch.cat([x, x.new_zeros(-x.numel() % 127)]).reshape(-1, 127)
        x = x * torch.where(torch.arange(x.shape[0])[:, None] % 2 == 0, 1.0, -1.0)
        rows.append(torch.cat([x, torch.full((x.shape[0], 1), top)], 1))
    x = torch.cat(rows).to(torch.bfloat16).cuda()[:, None]
    R = x.shape[0]
    c = _empty(1, R, 1, 128, fmt)
    ln = torch.zeros(1, dtype=torch.int32).cuda()
    _append(api, c, ln, x, -x, torch.zeros(R).cuda(), _cu([R]))
    for n, y in (("k", x), ("v", -x)):
        q, sc = ops_ref.quantise(y, fmt)
        assert torch.equal(c[n + "s"][0], sc)
        assert torch.equal(c[n + "c"][0].double(), q)


@pytest.mark.parametrize("fmt", FMTS)
def test_special_values(api, fmt):
    x = torch.randn(6, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x[0, 0, 5] = float("inf")
    x[1, 0, 6] = float("nan")
    x[2] = 0
    x[3] = x[3] * 2.0 ** -80        # below the smallest scale
    x[4] = torch.finfo(torch.bfloat16).max
    x[5] = x[5] * 2.0 ** -50
    c = _empty(1, 6, 1, 64, fmt)
    ln = torch.zeros(1, dtype=torch.int32).cuda()
    s = torch.tensor([1.0, float("-inf"), float("nan"), 0.0, -0.0, 2.0]).cuda()
    _append(api, c, ln, x, x, s, _cu([6]))
    _same({n: c[n] for n in ("kc", "ks", "sc")}, {n: _expect(_empty(1, 6, 1, 64, fmt), x, x, s, [6], [0])[n]
                                                  for n in ("kc", "ks", "sc")})
    k, v, so = api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, _cu([6]), 6)
    assert torch.isnan(k[:2]).all() and (k[2:4] == 0).all()
    assert torch.isfinite(k[4:]).all() and torch.equal(torch.nan_to_num(so), torch.nan_to_num(s))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,hkv,dh", [([1], 1, 64), ([5, 0, 9], 8, 128), ([130, 257], 3, 64)])
def test_read(api, fmt, dt, counts, hkv, dh):
    B, R, cap = len(counts), sum(counts), max(counts) + 4
    c = _empty(B, cap, hkv, dh, fmt, seed=5)
    first = [b % 3 for b in range(B)]
    ln = torch.tensor([n + 3 for n in counts], dtype=torch.int32).cuda()
    more = 3   # rows of the outputs behind the last sequence stay as they are
    out = (torch.full((R + more, hkv, dh), 9.0, dtype=dt).cuda(), torch.full((R + more, hkv, dh), 9.0, dtype=dt).cuda(),
           torch.full((R + more,), 9.0).cuda())
    k, v, s = api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, _cu(counts), R + more,
                                   start=torch.tensor(first, dtype=torch.int32).cuda(), out=out)
    for got, cc, sc in ((k, c["kc"], c["ks"]), (v, c["vc"], c["vs"])):
        want = torch.cat([cc[b, f:f + n].float() * sc[b, f:f + n, :, None] for b, (f, n) in enumerate(zip(first, counts))])
        assert torch.equal(got[:R], want.to(dt)) and (got[R:] == 9).all()
    assert torch.equal(s[:R], torch.cat([c["sc"][b, f:f + n] for b, (f, n) in enumerate(zip(first, counts))]))
    assert (s[R:] == 9).all()


def test_what_does_not_fit_is_left_and_recorded(api):
    CHECK = 7
    hkv, dh, cap = 2, 64, 10
    k, v, s = _rows(2, 9, hkv, dh)

    def run(start, cu, ln0, idx=None):
        c = _empty(3, cap, hkv, dh, torch.int8)
        ln = torch.tensor(ln0, dtype=torch.int32).cuda()
        before = {n: t.clone() for n, t in c.items()}
        _append(api, c, ln, k, v, s, torch.tensor(cu, dtype=torch.int32).cuda(), src_idx=idx,
                start=None if start is None else torch.tensor(start, dtype=torch.int32).cuda())
        st = api.device_status(reset=True)
        return before, c, ln.tolist(), st
    # the middle sequence is full: the others are written
    before, c, ln, st = run(None, [0, 3, 6, 9], [0, 8, 7])
    assert st == CHECK and ln == [3, 8, 10]
    _same(c, _expect(_expect(before, k, v, s, [3, 0, 0], [0, 0, 0]), k[6:], v[6:], s[6:], [0, 0, 3], [0, 0, 7]))
    for start, cu, ln0 in (([-1, 0, 0], [0, 3, 3, 3], [0, 0, 0]), (None, [3, 0, 0, 0], [0, 0, 0]),
                           (None, [0, 10, 10, 10], [0, 0, 0]), (None, [-2, 0, 0, 0], [5, 5, 5])):
        before, c, ln, st = run(start, cu, ln0)
        assert st == CHECK and ln[0] == ln0[0]
        _same({n: t[0] for n, t in c.items()}, {n: t[0] for n, t in before.items()})
    # a source row that is not there: zeros and score 0, the length still moves
    before, c, ln, st = run(None, [0, 1, 2, 3], [0, 0, 0], idx=torch.tensor([-1, 9, 4], dtype=torch.int32).cuda())
    assert st == CHECK and ln == [1, 1, 1]
    for b in (0, 1):
        assert (c["ks"][b, 0] == 0).all() and (c["kc"][b, 0] == 0).all() and c["sc"][b, 0] == 0
    # a read behind the length: that sequence's rows stay
    ln = torch.tensor([3, 2, 3], dtype=torch.int32).cuda()
    out = tuple(torch.full(sh, 5.0).cuda() for sh in ((9, hkv, dh), (9, hkv, dh), (9,)))
    api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, _cu([3, 3, 3]), 9, out=out)
    assert api.device_status(reset=True) == CHECK
    assert (out[0][3:6] == 5).all() and (out[2][3:6] == 5).all() and not (out[0][:3] == 5).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_stream_and_graph_replays(api, fmt):
    # an append in place, replayed: each replay adds the rows behind the ones before
    hkv, dh, cap, counts = 2, 128, 40, [3, 1]
    k, v, s = _rows(8, 4, hkv, dh)
    cu = _cu(counts)
    c = _empty(2, cap, hkv, dh, fmt)
    ln = torch.tensor([2, 5], dtype=torch.int32).cuda()
    want = _expect(_expect(c, k, v, s, counts, [2, 5]), k, v, s, counts, [5, 6])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    _append(api, c, ln, k, v, s, cu, stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _append(api, c, ln, k, v, s, cu)
        rd = api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, cu, 4)
    graph.replay()
    torch.cuda.synchronize()
    assert ln.tolist() == [8, 7]
    _same(c, want)
    assert torch.equal(rd[0][:3], (c["kc"][0, :3].float() * c["ks"][0, :3, :, None]).to(torch.bfloat16))


def test_many_sequences(api):
    # batches beyond one level of the sequence search, empty ones among them
    B, hkv, dh = 2500, 1, 64
    counts = [(b * 7) % 3 for b in range(B)]
    R = sum(counts)
    k, v, s = _rows(5, R, hkv, dh)
    c = _empty(B, 3, hkv, dh, torch.int8)
    ln = torch.zeros(B, dtype=torch.int32).cuda()
    _append(api, c, ln, k, v, s, _cu(counts))
    assert ln.tolist() == counts
    kr, _, sr = api.quant_cache_read(c["kc"], c["vc"], c["ks"], c["vs"], c["sc"], ln, _cu(counts), R,
                                     dtype=torch.float32)
    q, sc = ops_ref.quantise(k, torch.int8)
    assert torch.equal(kr, (q.float() * sc[..., None])) and torch.equal(sr, s)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_significand_against_every_maximum(api, fmt):
    # all 128 significands of a maximum, those of the values in 16 binades below it: every
    # quotient that can be a tie between two codes, and every one next to it
    x = torch.arange(128, 256, dtype=torch.float32)
    rows = []
    for top in range(128, 256):
        v = torch.cat([x[x <= top] * 2.0 ** -e for e in range(16)])
        v = torch.cat([v, v.new_zeros(-v.numel() % 127)]).reshape(-1, 127)
        rows.append(torch.cat([torch.full((v.shape[0], 1), float(top)), v], 1))
    x = torch.cat(rows).to(torch.bfloat16).cuda()[:, None]
    R = x.shape[0]
    for size in (1.0, 2.0 ** -40, 2.0 ** 90):
        y = (x.float() * size).to(torch.bfloat16)
        c = _empty(1, R, 1, 128, fmt)
        _append(api, c, torch.zeros(1, dtype=torch.int32).cuda(), y, -y, torch.zeros(R).cuda(), _cu([R]))
        for n, t in (("k", y), ("v", -y)):
            q, sc = ops_ref.quantise(t, fmt)
            assert torch.equal(c[n + "s"][0], sc)
            assert torch.equal(c[n + "c"][0].double(), q)
