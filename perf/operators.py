"""Cases for the operators around the quantised cache and drafted tokens.

Five operators: the per-head norm of queries and keys with the rotary embedding
(`rope`), its gradients (`rope_bwd`), writing rows into a quantised cache (`append`,
read back in the same pass so that what was stored comes out), reading a quantised
cache (`read`), and attention of a tree of drafted tokens over a cache (`tree`).

`run` computes an operator in plain torch when `own` is false and calls the framework
when it is true; `exact` is the operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

BASE = 1e6          # rotary base
EPS = 1e-6
DEV = "cuda"
MOST_BYTES = 190_000_000   # what a drawn case moves at most


# --------------------------------------------------------------------------- #
# cases                                                                       #
# --------------------------------------------------------------------------- #

def listed():
    return [
        # eight sequences generating: each one's new token, one row a sequence
        dict(name="rope step", op="rope", dtype="bf16", T=8, hq=16, hkv=8, dh=128, rot=128, packed=True),
        # a 16k prompt's rows, read as views of the packed projection output
        dict(name="rope prompt", op="rope", dtype="bf16", T=16384, hq=16, hkv=8, dh=128, rot=128, packed=True),
        # a training step on the kept rows of a 128k prompt
        dict(name="rope_bwd kept", op="rope_bwd", dtype="bf16", T=10721, hq=16, hkv=8, dh=128, rot=128, packed=False),
        # a gradient check's precision, wide heads that rotate only their first quarter
        dict(name="rope_bwd f32", op="rope_bwd", dtype="f32", T=1001, hq=8, hkv=2, dh=256, rot=64, packed=False),
        # the kept rows of eight ragged prompts enter an empty cache
        dict(name="append prompts", op="append", fmt="e4m3", B=8, rows=1868, cap=2048, hkv=8, dh=128, pick=False),
        # the accepted drafts of 16 sequences join their caches
        dict(name="append accepted", op="append", fmt="i8", B=16, rows=5, cap=4099, hkv=8, dh=128, pick=True),
        # a cache is read back in full for a second pass over its rows
        dict(name="read rows", op="read", fmt="i8", out="bf16", B=4, rows=10721, cap=10800, hkv=8, dh=128),
        # a few rows at full precision, as a check of a cache reads them
        dict(name="read few f32", op="read", fmt="e4m3", out="f32", B=3, rows=77, cap=300, hkv=4, dh=64),
        # one sequence's eight drafts over the cache a 16k prompt leaves
        dict(name="tree one prompt", op="tree", fmt="bf16", B=1, T=8, ragged=False, n=1868, cap=2048, hq=16, hkv=8, dh=128),
        # 32 sequences, one token each: plain decode over a quantised cache
        dict(name="tree single tokens", op="tree", fmt="e4m3", B=32, T=1, ragged=False, n=1868, cap=1900, hq=16, hkv=8, dh=128),
        # eight sequences of different lengths, up to what a 128k prompt leaves, 13 drafts at most
        dict(name="tree ragged", op="tree", fmt="bf16", B=8, T=13, ragged=True, n=10721, cap=10737, hq=16, hkv=8, dh=128),
        # the widest tree over two long caches, eight query heads a KV head
        dict(name="tree wide long", op="tree", fmt="i8", B=2, T=64, ragged=False, n=65500, cap=65600, hq=32, hkv=4, dh=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "read", "tree", "tree"])
    if op in ("rope", "rope_bwd"):
        dh = rng.choice([64, 128, 128, 256, 96])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4])
        rot = rng.choice([dh, dh, dh // 2 // 8 * 8, 16])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        row = (hq + hkv) * dh * (2 if dtype == "bf16" else 4) * (3 if op == "rope_bwd" else 2)
        return dict(op=op, dtype=dtype, T=_log(rng, 1, min(16384, MOST_BYTES // row)), hq=hq, hkv=hkv, dh=dh, rot=rot,
                    packed=rng.random() < 0.5)
    fmt = rng.choice(["i8", "e4m3"])
    dh = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    B = _log(rng, 1, 32)
    if op == "append":
        pick = rng.random() < 0.5
        rows = _log(rng, 1, 64 if pick else 1 + min(20000, MOST_BYTES // (hkv * dh * 12)) // B)
        return dict(op=op, fmt=fmt, B=B, rows=rows, cap=rows + _log(rng, 1, 2000), hkv=hkv, dh=dh, pick=pick)
    if op == "read":
        out = rng.choice(["bf16", "f32"])
        rows = _log(rng, 1, 1 + min(40000, MOST_BYTES // (hkv * dh * (6 if out == "bf16" else 10))) // B)
        return dict(op=op, fmt=fmt, out=out, B=B, rows=rows, cap=rows + rng.randrange(1, 200),
                    hkv=hkv, dh=dh)
    fmt = rng.choice(["bf16", "i8", "e4m3"])
    G = rng.choice([1, 2, 3, 4, 8])
    T = _log(rng, 1, 64)
    most = min(65500, 2 * 64 * 8 * 4 * 65500 // (B * T * G * hkv), MOST_BYTES // (B * hkv * 4 * dh))
    n = _log(rng, 1, max(1, most))
    return dict(op=op, fmt=fmt, B=B, T=T, ragged=rng.random() < 0.6, n=n, cap=n + rng.randrange(0, 100), hq=G * hkv,
                hkv=hkv, dh=dh)


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _counts(case):
    """Rows of each sequence: ragged, fixed by the case's sizes."""
    r = random.Random("%(op)s %(B)d %(rows)d" % case)
    return [case["rows"] if b == 0 else r.randint(max(0, case["rows"] // 2), case["rows"]) for b in range(case["B"])]


def _lens(case):
    """Cache lengths and drafted tokens of each sequence."""
    r = random.Random("%(B)d %(T)d %(n)d" % case)
    lens = [case["n"] if b == 0 or not case["ragged"] else r.randint(0, case["n"]) for b in range(case["B"])]
    dl = [case["T"] if b == 0 or not case["ragged"] else r.randint(1, case["T"]) for b in range(case["B"])]
    return lens, dl


# --------------------------------------------------------------------------- #
# inputs                                                                      #
# --------------------------------------------------------------------------- #

def _kv_rows(g, shape):
    """Key or value rows: unit normal with a few strong channels, as real keys have."""
    x = torch.randn(shape, generator=g, device=DEV)
    ch = torch.ones(shape[-2:], device=DEV)
    ch[:, torch.randint(0, shape[-1], (3,), generator=g, device=DEV)] = 6.0
    return (x * ch).to(torch.bfloat16)


def _store(x, fmt):
    """Rows as a quantised cache holds them: codes and scales."""
    qmax = 127.0 if fmt == "i8" else 448.0
    x = x.float()
    scale = x.abs().amax(-1) / qmax
    q = x / scale.clamp_min(1e-30)[..., None]
    code = torch.round(q).to(torch.int8) if fmt == "i8" else q.clamp(-448, 448).to(torch.float8_e4m3fn)
    return code, scale


def _tree_mask(T, seed):
    """Bit j of entry t: drafted token j is t itself or one of its ancestors."""
    r = random.Random(seed)
    bits = []
    for t in range(T):
        parent = -1 if t == 0 else r.randint(max(-1, t - 6), t - 1)
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << t)
    return [b - (1 << 64) if b >> 63 else b for b in bits]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(counts):
    c = [0]
    for n in counts:
        c.append(c[-1] + n)
    return _i32(c)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, st = case["op"], dict(case)
    if op in ("rope", "rope_bwd"):
        T, hq, hkv, dh, dt = case["T"], case["hq"], case["hkv"], case["dh"], _dt(case["dtype"])
        if case["packed"]:
            qkv = torch.randn(T, hq + 2 * hkv, dh, generator=g, device=DEV).mul_(1.7).to(dt)
            st["q"], st["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        else:
            st["q"] = torch.randn(T, hq, dh, generator=g, device=DEV).mul_(1.7).to(dt)
            st["k"] = torch.randn(T, hkv, dh, generator=g, device=DEV).mul_(0.6).to(dt)
        st["wq"] = 0.5 + torch.rand(dh, generator=g, device=DEV)
        st["wk"] = 0.5 + torch.rand(dh, generator=g, device=DEV)
        # kept rows sit anywhere in a 128k prompt, in order
        st["pos"] = torch.sort(torch.randint(0, 131072, (T,), generator=g, device=DEV))[0].to(torch.int32)
        if op == "rope_bwd":
            st["dq"] = torch.randn(T, hq, dh, generator=g, device=DEV).to(dt)
            st["dk"] = torch.randn(T, hkv, dh, generator=g, device=DEV).to(dt)
            if own:
                from learned_token_pruning_gemm_b200 import api
                st["ws"] = torch.empty(api.qk_norm_rope_bwd_workspace_size(T, hq, hkv, dh), dtype=torch.uint8,
                                       device=DEV)
        return st
    B, hkv, dh, cap = case["B"], case["hkv"], case["dh"], case["cap"]
    fmt = case["fmt"]
    code_t = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn, "bf16": torch.bfloat16}[fmt]
    if op == "append":
        counts = _counts(case)
        total = sum(counts)
        if case["pick"]:   # the accepted ones among the drafted rows
            src = 4 * total + 3
            st["idx"] = torch.sort(torch.randperm(src, generator=g, device=DEV)[:total])[0].to(torch.int32)
        else:
            src, st["idx"] = total, None
        st["k"], st["v"] = _kv_rows(g, (src, hkv, dh)), _kv_rows(g, (src, hkv, dh))
        st["s"] = torch.randn(src, generator=g, device=DEV)
        st["cu"], st["total"] = _cu(counts), total
        st["start"] = _i32([int(x) for x in torch.randint(0, cap - case["rows"] + 1, (B,), generator=g, device=DEV)])
        st["kc"] = torch.zeros(B, cap, hkv, dh, dtype=torch.int8, device=DEV).view(code_t)
        st["vc"] = torch.zeros(B, cap, hkv, dh, dtype=torch.int8, device=DEV).view(code_t)
        st["ks"] = torch.zeros(B, cap, hkv, device=DEV)
        st["vs"] = torch.zeros(B, cap, hkv, device=DEV)
        st["sc"] = torch.zeros(B, cap, device=DEV)
        st["len"] = st["start"].clone()
        return st
    kc, vc = _kv_rows(g, (B, cap, hkv, dh)), _kv_rows(g, (B, cap, hkv, dh))
    st["sc"] = torch.randn(B, cap, generator=g, device=DEV) * 2
    st["ks"] = st["vs"] = None
    if fmt != "bf16":
        kc, st["ks"] = _store(kc, fmt)
        vc, st["vs"] = _store(vc, fmt)
    st["kc"], st["vc"] = kc, vc
    if op == "read":
        counts = _counts(case)
        st["cu"], st["total"] = _cu(counts), sum(counts)
        st["len"] = _i32([n + (cap - case["rows"]) // 2 for n in counts])
        return st
    lens, dl = _lens(case)
    T, hq = case["T"], case["hq"]
    st["q"] = torch.randn(B, T, hq, dh, generator=g, device=DEV).to(torch.bfloat16)
    st["kd"], st["vd"] = _kv_rows(g, (B, T, hkv, dh)), _kv_rows(g, (B, T, hkv, dh))
    st["sd"] = torch.randn(B, T, generator=g, device=DEV)
    st["mask"] = torch.tensor([_tree_mask(T, "%d %d" % (seed, b)) for b in range(B)], dtype=torch.int64, device=DEV)
    st["len"], st["dl"] = _i32(lens), _i32(dl)
    st["gain"] = torch.rand(hq, generator=g, device=DEV)
    st["tau"] = 0.8 + 0.7 * torch.rand(hq, generator=g, device=DEV)
    st["out"] = torch.zeros(B, T, hq, dh, dtype=torch.bfloat16, device=DEV)
    if own:
        from learned_token_pruning_gemm_b200 import api
        st["ws"] = torch.empty(max(16, api.tree_attention_workspace_size(B, T, hq, hkv, dh, case["n"])),
                               dtype=torch.uint8, device=DEV)
    return st


# --------------------------------------------------------------------------- #
# the operators, plainly                                                      #
# --------------------------------------------------------------------------- #

def _angles(pos, rot):
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    a = pos.double()[:, None] * BASE ** (-2.0 * i / rot)
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _turn(x, cos, sin, rot):
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _plain_rope(st):
    cos, sin = _angles(st["pos"], st["rot"])
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        f = x.float()
        n = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w
        out.append(_turn(n, cos, sin, st["rot"]).to(x.dtype))
    return out


def _plain_rope_bwd(st):
    cos, sin = _angles(st["pos"], st["rot"])
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dq"]), (st["k"], st["wk"], st["dk"])):
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
        g = _turn(dy.float(), cos, -sin, st["rot"])
        xr = f * r
        dw.append((g * xr).sum((0, 1), dtype=torch.float64).float())
        wg = w * g
        dx.append((r * (wg - xr * (wg * xr).mean(-1, keepdim=True))).to(x.dtype))
    return dx + dw


def _round_e4m3(y):
    """To the nearest e4m3 value, ties to even, from 64 bits: four significant bits, or steps of 2^-9 below 2^-6."""
    b = y.view(torch.int64)
    b = (b + (2 ** 48 - 1) + ((b >> 49) & 1)) & -(2 ** 49)
    return torch.where(y.abs() < 2.0 ** -6, torch.round(y * 512.0) * 2.0 ** -9, b.view(torch.float64)).clamp(-448.0, 448.0)


def _plain_append(st):
    cu, B = st["cu"], st["B"]
    r = torch.arange(st["total"], device=DEV)
    b = torch.searchsorted(cu, r, right=True) - 1
    row = st["start"][b] + (r - cu[b])
    src = r if st["idx"] is None else st["idx"].long()
    read = []
    for x, c, s in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        f = x[src].float()
        scale = (f.abs().amax(-1).double() / (127.0 if st["fmt"] == "i8" else 448.0)).float()
        scale = torch.where(scale < 2.0 ** -60, 0.0, scale)
        y = f.double() / torch.where(scale == 0, 1.0, scale).double()[..., None]   # a border between two codes: 64 bits
        y = torch.where(scale[..., None] == 0, 0.0, y)
        y = torch.round(y).clamp(-127, 127) if st["fmt"] == "i8" else _round_e4m3(y)
        c[b, row] = y.to(c.dtype) if st["fmt"] == "i8" else y.float().to(c.dtype)
        s[b, row] = scale
        read.append((c[b, row].float() * s[b, row][..., None]).to(torch.bfloat16))
    st["sc"][b, row] = st["s"][src]
    st["len"].copy_(st["start"] + cu[1:] - cu[:-1])
    return read + [st["sc"][b, row], st["len"]]


def _plain_read(st):
    cu = st["cu"]
    r = torch.arange(st["total"], device=DEV)
    b = torch.searchsorted(cu, r, right=True) - 1
    row = r - cu[b]
    kv = [(c[b, row].float() * s[b, row][..., None]).to(_dt(st["out"]))
          for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]
    return kv + [st["sc"][b, row]]


def _plain_tree(st):
    B, T, hq, dh = st["q"].shape
    hkv, G, n = st["hkv"], hq // st["hkv"], st["n"]
    k, v = st["kc"][:, :n].float(), st["vc"][:, :n].float()
    if st["ks"] is not None:
        k, v = k * st["ks"][:, :n, :, None], v * st["vs"][:, :n, :, None]
    k, v = torch.cat([k, st["kd"].float()], 1), torch.cat([v, st["vd"].float()], 1)
    s = torch.cat([st["sc"][:, :n], st["sd"]], 1)
    q = st["q"].float().view(B, T, hkv, G, dh).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, dh)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, hkv, T, G, -1)
    z = z / (math.sqrt(dh) * st["tau"].view(1, hkv, 1, G, 1))
    z += st["gain"].view(1, hkv, 1, G, 1) * s[:, None, None, None]
    t = torch.arange(T, device=DEV)
    seen = torch.cat([(torch.arange(n, device=DEV) < st["len"][:, None])[:, None].expand(B, T, n),
                      ((st["mask"][..., None] >> t) & 1).bool() & (t < st["dl"][:, None])[:, None]], -1)
    z.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    p = (z - torch.where(m == float("-inf"), 0.0, m)).exp_()
    p /= p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(p.view(B, hkv, T * G, -1), v.permute(0, 2, 1, 3))
    o = o.view(B, hkv, T, G, dh).permute(0, 2, 1, 3, 4).reshape(B, T, hq, dh)
    return torch.where((t < st["dl"][:, None])[..., None, None], o, 0.0).to(torch.bfloat16)


# --------------------------------------------------------------------------- #
# the framework's calls                                                       #
# --------------------------------------------------------------------------- #

def _own(st):
    from learned_token_pruning_gemm_b200 import api
    op = st["op"]
    if op == "rope":
        return api.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["pos"], eps=EPS, rope_base=BASE,
                                rot_dim=st["rot"])
    if op == "rope_bwd":
        return api.qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["dq"], st["dk"], eps=EPS,
                                    rope_base=BASE, rot_dim=st["rot"], workspace=st["ws"])
    if op == "append":
        api.quant_cache_append(st["k"], st["v"], st["s"], st["cu"], st["kc"], st["vc"], st["ks"], st["vs"], st["sc"],
                               st["len"], start=st["start"], src_idx=st["idx"])
        k, v, s = api.quant_cache_read(st["kc"], st["vc"], st["ks"], st["vs"], st["sc"], st["len"], st["cu"],
                                       st["total"], start=st["start"])
        return k, v, s, st["len"]
    if op == "read":
        return api.quant_cache_read(st["kc"], st["vc"], st["ks"], st["vs"], st["sc"], st["len"], st["cu"], st["total"],
                                    dtype=_dt(st["out"]))
    return api.tree_attention(st["q"], st["kd"], st["vd"], st["sd"], st["mask"], st["kc"], st["vc"], st["sc"],
                              st["len"], st["gain"], st["tau"], st["n"], draft_len=st["dl"], k_scale=st["ks"],
                              v_scale=st["vs"], out=st["out"], workspace=st["ws"])


def run(st):
    if own:
        return _own(st)
    return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "append": _plain_append, "read": _plain_read,
            "tree": _plain_tree}[st["op"]](st)


# --------------------------------------------------------------------------- #
# what a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    op, dh, hkv = case["op"], case["dh"], case["hkv"]
    if op in ("rope", "rope_bwd"):
        n = case["T"] * (case["hq"] + hkv) * dh
        es = 2 if case["dtype"] == "bf16" else 4
        if op == "rope":
            return {"bytes": 2 * n * es + 4 * case["T"] + 8 * dh, "flops": 8 * n}
        return {"bytes": 3 * n * es + 4 * case["T"] + 16 * dh, "flops": 16 * n}
    if op in ("append", "read"):
        total = sum(_counts(case))
        stored = total * (hkv * 2 * (dh + 4) + 4)
        if op == "append":
            given = total * (hkv * 2 * dh * 2 + 4)
            return {"bytes": 2 * given + stored, "flops": 8 * total * hkv * dh}
        es = 2 if case["out"] == "bf16" else 4
        return {"bytes": stored + total * (hkv * 2 * dh * es + 4), "flops": 2 * total * hkv * dh}
    lens, dl = _lens(case)
    hq = case["hq"]
    row = hkv * 2 * dh * 2 if case["fmt"] == "bf16" else hkv * 2 * (dh + 4)
    b = sum(n * (row + 4) + t * (hkv * 2 * dh * 2 + 12 + 2 * hq * dh * 2) for n, t in zip(lens, dl))
    return {"bytes": b, "flops": sum(4 * dh * hq * t * (n + t) for n, t in zip(lens, dl))}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits                                                  #
# --------------------------------------------------------------------------- #

def _exact_norm(x, w, pos, rot):
    x = x.double()
    r = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).pow(-0.5)
    return x, r, w.double()


def _exact_rotate(y, pos, rot, sign):
    """Pairs (i, i + rot/2) as complex numbers, times exp(sign * i * angle)."""
    half = rot // 2
    freq = torch.exp(torch.arange(half, device=DEV, dtype=torch.float64) * (-2.0 / rot * math.log(BASE)))
    z = torch.complex(y[..., :half], y[..., half:rot])
    z = z * torch.polar(torch.ones_like(freq), sign * pos.double()[:, None] * freq)[:, None]
    return torch.cat([z.real, z.imag, y[..., rot:]], -1)


def _exact_codes(x, fmt):
    """(value, scale): the definition of what a row is stored as."""
    x = x.double()
    top = x.abs().max(-1).values
    scale = (top / torch.full_like(top, 127 if fmt == "i8" else 448)).float().double()   # scales are held in 32 bits
    scale[scale < 2.0 ** -60] = 0
    y = x / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)
    if fmt == "i8":
        code = y.round().clamp(-127, 127)
    else:   # the nearest of the format's values, the even code of two that are as near
        grid = torch.arange(127, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
        hi = torch.bucketize(y.abs(), grid).clamp_max(126)
        lo = (hi - 1).clamp_min(0)
        up, down = grid[hi] - y.abs(), y.abs() - grid[lo]
        code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo]) * y.sign()
    return torch.where(scale.unsqueeze(-1) > 0, code * scale.unsqueeze(-1), torch.zeros_like(code))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            x, r, w = _exact_norm(x, w, st["pos"], st["rot"])
            out.append(_exact_rotate(x * r * w, st["pos"], st["rot"], 1.0))
        return out
    if op == "rope_bwd":
        dx, dw = [], []
        for x, w, dy in ((st["q"], st["wq"], st["dq"]), (st["k"], st["wk"], st["dk"])):
            x, r, w = _exact_norm(x, w, st["pos"], st["rot"])
            g = _exact_rotate(dy.double(), st["pos"], st["rot"], -1.0)
            dw.append((g * x * r).sum(1).sum(0))
            h = g * w
            dx.append(r * h - r.pow(3) * x * ((h * x).sum(-1, keepdim=True) / x.shape[-1]))
        return dx + dw
    if op == "append":
        src = slice(None) if st["idx"] is None else st["idx"].long()
        kv = [_exact_codes(x[src], case["fmt"]) for x in (st["k"], st["v"])]
        return kv + [st["s"][src].double(), None]
    if op == "read":
        rows = [(b, n) for b, n in enumerate(_counts(case))]
        kv = [torch.cat([c[b, :n].double() * s[b, :n, :, None].double() for b, n in rows])
              for c, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]
        return kv + [torch.cat([st["sc"][b, :n].double() for b, n in rows])]
    lens, dl = _lens(case)
    B, T, hq, hkv, dh = case["B"], case["T"], case["hq"], case["hkv"], case["dh"]
    out = torch.zeros(B, T, hq, dh, dtype=torch.float64, device=DEV)
    masks = st["mask"].tolist()
    for b in range(B):
        n, t = lens[b], dl[b]
        bits = torch.tensor([[bool(m >> i & 1) for i in range(t)] for m in masks[b][:t]], device=DEV)
        for h in range(hkv):
            k, v = st["kc"][b, :n, h].double(), st["vc"][b, :n, h].double()
            if st["ks"] is not None:
                k, v = k * st["ks"][b, :n, h, None].double(), v * st["vs"][b, :n, h, None].double()
            k, v = torch.cat([k, st["kd"][b, :t, h].double()]), torch.cat([v, st["vd"][b, :t, h].double()])
            s = torch.cat([st["sc"][b, :n], st["sd"][b, :t]]).double()
            for i in range(hq // hkv):
                j = h * (hq // hkv) + i
                z = st["q"][b, :t, j].double() @ k.T / (dh ** 0.5 * st["tau"][j].double()) + st["gain"][j].double() * s
                z[:, n:][~bits] = -math.inf
                out[b, :t, j] = torch.softmax(z, -1) @ v
    return out

