"""Plain 64-bit forms of the q/k norm with rotation, the quantised cache and the
attention of drafted tokens, written from their formulas, one sequence and head at a
time where that is plainer. They run on whatever device their inputs are on and share
no code with the kernels."""
import math

import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


# ---- norm of q and k with the rotation ----

def rotation(pos, rot, base, dtype=torch.float64):
    """cos and sin [T, rot/2] of pos * base^(-2i/rot). The product is taken modulo one
    turn in integers of 2^-62 of a turn, so far positions keep 64-bit accuracy."""
    cos, sin = [], []
    for p in pos.tolist():
        c, s = [], []
        for i in range(rot // 2):
            f = int(math.ldexp(base ** (-2.0 * i / rot) / (2 * math.pi), 62))
            a = 2 * math.pi * (((p * f) % (1 << 62)) / (1 << 62))
            c.append(math.cos(a))
            s.append(math.sin(a))
        cos.append(c)
        sin.append(s)
    shape = (len(cos), 1, rot // 2)
    t = lambda v: torch.tensor(v, dtype=dtype, device=pos.device).reshape(shape)
    return t(cos), t(sin)


def rotate(x, cos, sin):
    h = cos.shape[-1]
    a, b, rest = x[..., :h], x[..., h:2 * h], x[..., 2 * h:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def norm_rope(x, w, cos, sin, eps):
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return rotate(x * r * w.double(), cos, sin)


def pair_size(x, cos):
    """|x_i| + |x_{i + rot/2}| in both places of a rotated pair (what a rotation's rounding
    errors are relative to), |x| elsewhere."""
    h = cos.shape[-1]
    a, b, rest = x[..., :h].abs(), x[..., h:2 * h].abs(), x[..., 2 * h:].abs()
    return torch.cat([a + b, a + b, rest], -1)


def norm_rope_bwd(x, w, cos, sin, eps, dy):
    """(dx, dw, size of dx's terms, size of dw's terms)."""
    x, w, dy = x.double(), w.double(), dy.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g = rotate(dy, cos, -sin)
    gs = pair_size(dy, cos)
    xr = x * r
    wg = w * g
    dx = r * (wg - xr * (wg * xr).mean(-1, keepdim=True))
    size = r * (w.abs() * gs + xr.abs() * (w.abs() * gs * xr.abs()).mean(-1, keepdim=True))
    return dx, (g * xr).sum((0, 1)), size, (gs * xr.abs()).sum((0, 1))


# ---- quantised rows ----

def e4m3_values():
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def quantise(x, code_dtype):
    """(codes as values [..., dh] f64, scale [...] f32) of bf16 rows."""
    x = x.double()
    scale = (x.abs().amax(-1) / QMAX[code_dtype]).float()
    bad = ~torch.isfinite(x).all(-1)
    scale[scale < 2.0 ** -60] = 0.0
    scale[bad] = float("nan")
    s = torch.where(scale > 0, scale.double(), torch.ones_like(scale.double()))
    y = torch.where((scale > 0)[..., None], x / s[..., None], torch.zeros_like(x))
    if code_dtype == torch.int8:
        return torch.round(y).clamp(-127, 127), scale
    grid = e4m3_values().to(x.device)
    hi = torch.bucketize(y.abs().contiguous(), grid).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - y.abs(), y.abs() - grid[lo]
    mag = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
    return torch.where(y < 0, -mag, mag), scale


# ---- drafted tokens over a cache ----

def tree_attention(q, kd, vd, sd, mask, k, v, s, lens, dls, gain, tau):
    """(out, spread) [B,T,Hq,dh] f64 from the cache's values k, v [B,cap,Hkv,dh]; rows that
    are not drafted stay NaN. spread is sum_j p_j |v_j - out|, what relative errors of the
    weights act on."""
    B, T, hq, dh = q.shape
    G = hq // k.shape[2]
    out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
    spread = out.clone()
    for b in range(B):
        n, dl = int(lens[b]), int(dls[b])
        for t in range(dl):
            m = int(mask[b, t]) & ((1 << 64) - 1)
            see = [i for i in range(dl) if m >> i & 1]
            ss = torch.cat([s[b, :n], sd[b, see]]).double()
            for h in range(hq):
                kk = torch.cat([k[b, :n, h // G].double(), kd[b, see, h // G].double()])
                vv = torch.cat([v[b, :n, h // G].double(), vd[b, see, h // G].double()])
                z = kk @ q[b, t, h].double() / (math.sqrt(dh) * float(tau[h])) + float(gain[h]) * ss
                if z.numel() == 0 or (z == -math.inf).all():
                    out[b, t, h] = 0.0
                    spread[b, t, h] = 0.0
                    continue
                p = torch.exp(z - z.max())
                p = p / p.sum()
                p, vv = p[p > 0], vv[p > 0]
                o = p @ vv
                out[b, t, h] = o
                spread[b, t, h] = p @ (vv - o).abs()
    return out, spread
