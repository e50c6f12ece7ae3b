"""GPU parity of tg_tree_attention against the 64-bit form of ops_ref.py.

Tolerance, per element: the output is stored in bf16 (half a step: 2^-8 of it). The
weights p_j are rounded to bf16 before the product with the values, and the row's sum
adds the rounded ones, so relative errors e_j <= 2^-8 move the output by at most
sum p_j |e_j| |v_j - out| / (1 - 2^-8): 2^-8 of the spread that ops_ref gives. What is
left is fp32: logits off by about 2^-22 of sum |q k| c (below 2^8 here) and the
exponential's 2^-22: 2^-12 of the spread covers them.

Over a cache of codes the weights are rounded to fp16 (2^-11) and the row's sum adds them
as they were: the output moves by at most 2^-11 sum p_j |v_j|, where |v_j| <= |out| +
|v_j - out|. Of the spread that is less than the bound above; 2^-11 |out| comes on top of
it (a row of one key is off by its weight's rounding), which reference() adds as 2^-8 of
|out| / 8."""
import pytest
import torch

import ops_ref

pytestmark = pytest.mark.gpu
BF, I8, E4 = torch.bfloat16, torch.int8, torch.float8_e4m3fn


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


def make(seed, B, T, cap, lens, hq, hkv, dh, fmt, dls=None, garbage=True):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    st = dict(q=rnd(B, T, hq, dh).to(BF), kd=rnd(B, T, hkv, dh).to(BF), vd=rnd(B, T, hkv, dh).to(BF),
              sd=rnd(B, T), sc=rnd(B, cap) * 2, gain=torch.rand(hq, generator=g),
              tau=0.8 + 0.7 * torch.rand(hq, generator=g))
    k, v = rnd(B, cap, hkv, dh).to(BF), rnd(B, cap, hkv, dh).to(BF)
    parents = [[-1 if t == 0 else int(torch.randint(max(-1, t - 5), t, (1,), generator=g)) for t in range(T)]
               for _ in range(B)]
    from learned_token_pruning_gemm_b200 import api
    st["mask"] = api.tree_mask(parents)
    st["len"] = torch.tensor(lens, dtype=torch.int32)
    st["dl"] = torch.tensor(dls if dls is not None else [T] * B, dtype=torch.int32)
    if fmt == BF:
        st["kc"], st["vc"], st["ks"], st["vs"] = k, v, None, None
    else:
        for n, x in (("k", k), ("v", v)):
            code, scale = ops_ref.quantise(x, fmt)
            st[n + "c"], st[n + "s"] = code.float().to(fmt), scale
    if garbage:   # rows behind the cache's end and drafts that are not there hold anything
        for b in range(B):
            n, dl = lens[b], int(st["dl"][b])
            st["sc"][b, n:] = float("nan")
            if fmt == BF:
                st["kc"][b, n:] = float("nan")
                st["vc"][b, n:] = float("inf")
            else:
                st["ks"][b, n:] = float("nan")
                st["vs"][b, n:] = float("inf")
            st["kd"][b, dl:] = float("nan")
            st["vd"][b, dl:] = float("nan")
            st["sd"][b, dl:] = float("inf")
            st["mask"][b, :dl] |= ~0 << dl if dl < 64 else 0   # bits of drafts that are not there
            st["q"][b, dl:] = float("nan")
    return {n: None if t is None else t.cuda() for n, t in st.items()}


def values(st):
    if st["ks"] is None:
        return st["kc"].double(), st["vc"].double()
    return st["kc"].double() * st["ks"].double()[..., None], st["vc"].double() * st["vs"].double()[..., None]


def run(api, st, out=None, max_len=None, **kw):
    ml = int(st["len"].max()) if max_len is None else max_len
    return api.tree_attention(st["q"], st["kd"], st["vd"], st["sd"], st["mask"], st["kc"], st["vc"], st["sc"],
                              st["len"], st["gain"], st["tau"], ml, draft_len=st["dl"], k_scale=st["ks"],
                              v_scale=st["vs"], out=out, **kw)


def reference(st):
    k, v = values(st)
    out, spread = ops_ref.tree_attention(st["q"], st["kd"], st["vd"], st["sd"], st["mask"].cpu(), k, v, st["sc"],
                                         st["len"].cpu(), st["dl"].cpu(), st["gain"].cpu(), st["tau"].cpu())
    return out, spread if st["ks"] is None else spread + out.abs() / 8


def check(got, ref, keep=9.0):
    want, spread = ref
    there = ~torch.isnan(want)
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -7) + (2.0 ** -8 + 2.0 ** -7 * 2.0 ** -8 + 2.0 ** -12) * spread + 1e-6
    err = (got.double() - want).abs()
    bad = there & ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} of {int(there.sum())} outside, worst {float((err / tol)[bad].max()):.2f} "
                           f"at {bad.nonzero()[0].tolist()}: {float(got[bad][0])} for {float(want[bad][0])}")
    if keep is not None:
        assert (got[~there] == keep).all(), "rows that are not drafted were written"
    return float((err / tol)[there].max()) if there.any() else 0.0


CASES = [  # B, T, cap, lens, hq, hkv, dh, dls
    (1, 1, 1, [0], 2, 1, 128, None),                      # nothing cached: only itself
    (2, 1, 300, [257, 1], 16, 8, 128, None),              # single tokens
    (3, 5, 200, [128, 0, 127], 4, 2, 128, [5, 3, 0]),     # tile edges, an empty cache, no drafts
    (2, 64, 150, [129, 40], 4, 1, 128, [64, 33]),         # 256 rows a KV head
    (1, 13, 1900, [1868], 16, 8, 128, None),
    (2, 9, 500, [500, 131], 6, 2, 64, [9, 1]),            # groups of three, head dim 64
    (1, 40, 260, [260], 8, 1, 64, [37]),                  # groups of eight
    (2, 17, 90, [64, 90], 20, 1, 128, [17, 16]),          # a group of twenty
    (1, 2, 140, [140], 128, 1, 64, None),                 # a group of 128
    (9, 3, 700, [700, 1, 0, 333, 64, 65, 512, 130, 699], 8, 4, 128, [3, 2, 1, 3, 0, 3, 1, 2, 3]),
    (40, 2, 90, [(7 * b) % 91 for b in range(40)], 8, 8, 128, None),
]


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("B,T,cap,lens,hq,hkv,dh,dls", CASES)
def test_against_the_64_bit_form(api, fmt, B, T, cap, lens, hq, hkv, dh, dls):
    st = make(B * 100 + T, B, T, cap, lens, hq, hkv, dh, fmt, dls)
    out = torch.full_like(st["q"], 9.0)
    got = run(api, st, out=out)
    assert got is out
    worst = check(out, reference(st))
    print(f"worst error {worst:.2f} of the tolerance")
    again = run(api, st, out=torch.full_like(out, 9.0))
    assert torch.equal(again, out), "a fixed order of sums"


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_longer_bound_than_lengths(api, fmt):
    # max_len is only a bound: the split that it sizes must not change what is attended
    st = make(3, 3, 4, 2000, [700, 1, 130], 8, 2, 128, fmt)
    ref = reference(st)
    for ml in (700, 1024, 2000):
        check(run(api, st, out=torch.full_like(st["q"], 9.0), max_len=ml), ref)


@pytest.mark.parametrize("fmt", [BF, E4])
def test_long_cache(api, fmt):
    st = make(11, 1, 3, 20000, [19999], 4, 2, 128, fmt, garbage=False)
    check(run(api, st), reference(st), keep=None)


def test_masks(api):
    # any set of bits: nothing, later tokens, all; over an empty and a short cache
    st = make(5, 2, 6, 40, [0, 40], 4, 2, 128, BF, garbage=False)
    st["mask"][:, 0] = 0
    st["mask"][:, 1] = 1 << 5
    st["mask"][:, 2] = 63
    st["mask"][:, 3] = -1
    got = run(api, st)
    check(got, reference(st))
    assert (got[0, 0] == 0).all()


@pytest.mark.parametrize("fmt", [BF, I8])
def test_scores_of_minus_infinity(api, fmt):
    st = make(6, 2, 3, 200, [150, 20], 4, 2, 128, fmt, garbage=False)
    st["gain"].fill_(0.5)
    st["sc"][0, ::2] = float("-inf")
    st["sc"][1] = float("-inf")
    st["sd"][1] = float("-inf")
    got = run(api, st)
    check(got, reference(st))
    assert (got[1] == 0).all()
    st["sc"][0] = torch.finfo(torch.float32).min   # the type's lowest value: everything else outweighs it
    st["sd"][0] = 1.0
    check(run(api, st), reference(st))


@pytest.mark.parametrize("fmt", [BF, I8, E4])
def test_hidden_infinities_and_nan_do_not_spread(api, fmt):
    # drafts 2 and 4 hold NaN and infinities; only the tokens that see them show it
    st = make(7, 1, 6, 100, [77], 4, 2, 128, fmt, garbage=False)
    st["mask"][0] = torch.tensor([1, 3, 7, 8 | 1, 16, 32 | 1]).cuda()
    clean = run(api, st)
    st["kd"][0, 2] = float("nan")
    st["vd"][0, 2, :, ::7] = float("nan")
    st["vd"][0, 4, :, 3] = float("inf")
    st["vd"][0, 4, 1, 9] = float("-inf")
    got = run(api, st)
    for t in (0, 1, 3, 5):
        assert torch.equal(got[0, t], clean[0, t])
    assert torch.isnan(got[0, 2]).all()
    inf = got[0, 4].float()
    assert (inf[:, 3] == float("inf")).all() and (inf[2:, 9] == float("-inf")).all()
    others = torch.ones(128, dtype=torch.bool)
    others[[3, 9]] = False
    assert torch.equal(got[0, 4, :, others], clean[0, 4, :, others])
    assert torch.equal(got[0, 4, :2, 9], clean[0, 4, :2, 9])
    # a visible NaN key or an infinite visible logit is seen
    st = make(7, 1, 6, 100, [77], 4, 2, 128, fmt, garbage=False)
    st["sc"][0, 30] = float("nan")
    assert torch.isnan(run(api, st)).all()


@pytest.mark.parametrize("fmt", [BF, I8])
def test_dominant_and_flat_logits(api, fmt):
    # logits that grow along the cache move the running maximum at every tile; a key far
    # ahead of the others takes its whole row
    st = make(8, 1, 4, 900, [900], 4, 2, 128, fmt, garbage=False)
    st["gain"].fill_(1.0)
    st["sc"][0] = torch.arange(900, dtype=torch.float32).cuda() * 0.25 - 60
    check(run(api, st), reference(st), keep=None)
    st["sc"][0] = 60 - torch.arange(900, dtype=torch.float32).cuda() * 0.25
    check(run(api, st), reference(st), keep=None)
    st["sc"][0] = 0
    st["sc"][0, 123] = 200
    check(run(api, st), reference(st), keep=None)
    st["gain"].zero_()
    st["q"].zero_()
    check(run(api, st), reference(st), keep=None)


def test_single_token_matches_decode(api):
    # one drafted token with mask 1 is decode of a token whose row is appended first
    B, cap, hq, hkv = 3, 300, 16, 8
    st = make(9, B, 1, cap, [299, 64, 0], hq, hkv, 128, BF, garbage=False)
    got = run(api, st, max_len=299)
    ln = st["len"].clone()
    api.cache_append(st["kd"][:, 0].contiguous(), st["vd"][:, 0].contiguous(), st["sd"][:, 0].contiguous(),
                     st["kc"], st["vc"], st["sc"], ln)
    want = api.gated_decode(st["q"][:, 0].contiguous(), st["kc"], st["vc"], st["sc"], ln, st["gain"], st["tau"], cap)
    check(got[:, 0].unsqueeze(1), (want.double().unsqueeze(1), torch.ones_like(want, dtype=torch.float64).unsqueeze(1)),
          keep=None)


def test_bad_lengths_are_skipped_and_recorded(api):
    st = make(10, 4, 3, 100, [100, 50, 60, 20], 4, 2, 128, BF, garbage=False)
    ref = reference(st)
    for ln, dl in (([100, -1, 60, 20], [3, 3, 3, 3]), ([100, 101, 60, 20], [3, 3, 3, 3]),
                   ([100, 50, 60, 20], [3, 4, 3, 3]), ([100, 50, 60, 20], [3, -1, 3, 3])):
        bad = dict(st, len=torch.tensor(ln, dtype=torch.int32).cuda(), dl=torch.tensor(dl, dtype=torch.int32).cuda())
        out = torch.full_like(st["q"], 9.0)
        run(api, bad, out=out, max_len=100)
        assert api.device_status(reset=True) == 7
        assert (out[1] == 9).all()
        keep = [0, 2, 3]
        check(out[keep], (ref[0][keep], ref[1][keep]))


@pytest.mark.parametrize("fmt", [BF, E4])
def test_streams_and_graphs(api, fmt):
    # two calls at once on two streams, each with its own workspace; then one graph whose
    # replay follows lengths that change on the device
    a = make(21, 2, 5, 400, [400, 31], 8, 2, 128, fmt, garbage=False)
    b = make(22, 1, 8, 1500, [1444], 8, 4, 128, fmt, garbage=False)
    ra, rb = reference(a), reference(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa = [run(api, a, stream=s1, max_len=400) for _ in range(3)]
    ob = [run(api, b, stream=s2, max_len=1500) for _ in range(3)]
    torch.cuda.synchronize()
    for o in oa:
        check(o, ra, keep=None)
    for o in ob:
        check(o, rb, keep=None)
    out = torch.full_like(a["q"], 9.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(api, a, out=out, max_len=400)
    a["len"].copy_(torch.tensor([17, 399], dtype=torch.int32))
    a["dl"].copy_(torch.tensor([5, 2], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(out, reference(a))


def test_no_sequences_and_no_drafts(api):
    st = make(1, 1, 2, 10, [5], 4, 2, 128, BF)
    e = {n: t if t is None or n in ("gain", "tau") else t[:0] for n, t in st.items()}
    assert run(api, e, max_len=5).shape == (0, 2, 4, 128)
    e = {n: t[:, :0].contiguous() if n in ("q", "kd", "vd", "sd", "mask") else t for n, t in st.items()}
    e["dl"] = e["dl"] * 0
    assert run(api, e).shape == (1, 0, 4, 128)


EDGES = [  # rows around the tiles of the few-row kernel, heads it cannot share evenly; pairs of row tiles
    (2, 8, 300, [300, 17], 3, 3, 128, [8, 7]),
    (2, 9, 300, [299, 16], 5, 5, 128, None),
    (1, 8, 700, [700], 24, 12, 128, None),
    (2, 17, 333, [333, 15], 12, 12, 128, [17, 16]),
    (3, 64, 400, [400, 192, 193], 5, 1, 128, [64, 44, 20]),     # three row tiles, two, one
    (2, 64, 400, [65, 64], 10, 2, 64, [64, 23]),
    (4, 64, 90, [1, 90, 64, 65], 2, 1, 128, [64, 64, 63, 1]),   # one full row tile: units with and without a second half
    (5, 64, 2000, [2000, 3, 1999, 0, 640], 12, 3, 128, [64, 64, 1, 9, 43]),
    (64, 3, 400, [(53 * b) % 401 for b in range(64)], 16, 8, 64, None),   # more items than CTAs
]


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("B,T,cap,lens,hq,hkv,dh,dls", EDGES)
def test_edges(api, fmt, B, T, cap, lens, hq, hkv, dh, dls):
    st = make(B * 100 + T + 7, B, T, cap, lens, hq, hkv, dh, fmt, dls)
    check(run(api, st, out=torch.full_like(st["q"], 9.0)), reference(st))


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("T,hq,dh", [(2, 4, 128), (40, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 40, 2.0 ** 80])
def test_logits_whose_last_place_exceeds_any_weight(api, fmt, T, hq, dh, size):
    # Logits of this size differ by far more than a softmax tells apart: every row is its
    # best key's value, and nothing may be lost in taking the reference off. The best
    # key is ahead by more than the logits' rounding (2^-20 of the largest).
    st = make(31, 1, T, 600, [577], hq, 2, dh, fmt, garbage=False)
    st["q"] = (st["q"].float() * size).to(BF)
    st["gain"].zero_()
    st["mask"][:] = 0
    k, v = values(st)
    z = torch.einsum("tghd,ngd->tghn", st["q"][0].double().reshape(T, 2, hq // 2, dh), k[0, :577])
    top = z.topk(2, -1)
    ahead = (top.values[..., 0] - top.values[..., 1]) > z.abs().amax(-1) * 2.0 ** -17
    assert ahead.float().mean() > 0.9
    want = torch.einsum("tghn,ngd->tghd", torch.nn.functional.one_hot(top.indices[..., 0], 577).double(), v[0, :577])
    got = run(api, st)[0].double().reshape(T, 2, hq // 2, dh)
    assert torch.isfinite(got).all()
    err = (got - want).abs()[ahead]
    assert (err <= want.abs()[ahead] * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12)).all(), float(err.max())


@pytest.mark.parametrize("fmt", [BF, I8, E4])
@pytest.mark.parametrize("T,hq,hkv,dh", [(64, 24, 6, 128), (64, 24, 6, 64), (2, 12, 12, 128), (20, 8, 4, 128)])
def test_the_same_bits_every_time(api, fmt, T, hq, hkv, dh):
    # a tile given back too early is overwritten now and then only: many calls in a row
    st = make(5, 3, T, 3100, [2844, 3100, 1251], hq, hkv, dh, fmt)
    want = run(api, st, out=torch.full_like(st["q"], 9.0))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    out = torch.empty_like(want)
    for _ in range(1000):
        out.fill_(9.0)
        differ += (run(api, st, out=out) != want).any()
    assert int(differ) == 0
