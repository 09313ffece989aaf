"""The gated recurrence in 64 bits, one step after another, forward and backward, each value with a bound
on what fp32 arithmetic may be off by.

The bounds count roundings as in serving_ref.py: U = 2^-24 is the largest relative error of one fp32
rounding; a hardware exp2, reciprocal or square root is taken as 2 U.  `ev` are absolute errors, `rv`
relative ones.  The kernels compose stretches of rows: a value that passes n rows meets one rounding a row
and one for each of the 8-row parts that it passes, at most two a row, and six more where a stretch is cut
short and joined (the lane's, the part's, the tile's map and their products)."""
from __future__ import annotations

import torch

from serving_ref import U, check, f64, half_step, silu  # noqa: F401


def sigmoid(v, mag):
    """(sigmoid(v), its relative error): v is a sum of parts of size mag, rounded once; the exponent v log2(e)
    is rounded twice more, its factor e^-v weighs at most 1 in 1 + e^-v; exp2, sum and reciprocal 5 U.  An
    infinite v rounds nowhere: 1 + e^-v is 1 or infinite."""
    s = torch.sigmoid(v)
    mag = torch.where(mag.isinf(), 0.0, mag)
    return s, (5 + 3 * mag * (1 - s)) * U


def gates(x, ag, xg, param, ab, xb, scale):
    """Everything of a step but the recurrence, elementwise, with relative errors."""
    ab, xb = (torch.zeros_like(param) if t is None else t for t in (ab, xb))
    r, rr = sigmoid(ag + ab, ag.abs() + ab.abs())
    i, ri = sigmoid(xg + xb, xg.abs() + xb.abs())
    sp = torch.nn.functional.softplus(param, threshold=1e9)
    l = -scale * sp * r
    # the library's exp and log1p and a sum: softplus is off by at most 8 U, two products more
    rl = rr + 10 * U
    a = torch.exp(l)
    ra = l.abs() * (rl + 2 * U) + 2 * U
    w2 = -torch.expm1(2 * l)
    # a relative error of l moves 1 - a^2 by at most as much; the series and its product 8 U.  The difference
    # from p = -2 l = 0.35 on: a^2's error and its rounding over what is left of 1
    rest = (2 * a * a * ra + 2 * U) / w2.clamp(min=1e-300)
    rw = torch.where(-2 * l < 0.3499, rl + 8 * U, torch.where(-2 * l > 0.3501, rest, (rl + 8 * U).maximum(rest)))
    w = torch.sqrt(w2)
    rw = rw / 2 + 2 * U
    q = torch.where(w > 0, -l * a * a / w.clamp(min=1e-300), 0.0)
    rq = rl + 2 * ra + rw + 6 * U
    return dict(x=x, r=r, rr=rr, i=i, ri=ri, l=l, rl=rl, a=a, ra=ra, w=w, rw=rw, q=q, rq=rq, u=i * x, ru=ri + U,
                b=w * i * x, rb=rw + ri + 2 * U, ratio=torch.sigmoid(param) / sp.clamp(min=1e-300))


def run(g, h0):
    """States h (L, ...) and their bounds from gates laid out (L, ...)."""
    h, e, m = h0.clone(), torch.zeros_like(h0), h0.abs()
    hs, es = [], []
    for t in range(g["a"].shape[0]):
        a, b = g["a"][t], g["b"][t]
        e = a * e + a * m * g["ra"][t] + b.abs() * g["rb"][t]
        h, m = a * h + b, a * m + b.abs()
        e = e + 2 * U * m
        hs.append(h)
        es.append(e + 6 * U * m)
    if not hs:
        return h0.new_zeros((0,) + h0.shape), h0.new_zeros((0,) + h0.shape)
    return torch.stack(hs), torch.stack(es)


def forward(x, ag, xg, param, ab=None, xb=None, z=None, scale=8.0, h0=None):
    """x, ag, xg, z (L, ...) in 64 bits with the channels last; y, its bound, the states and theirs."""
    g = gates(x, ag, xg, param, ab, xb, scale)
    h, e = run(g, x.new_zeros(x.shape[1:]) if h0 is None else h0)
    if z is None:
        return h, e, h, e
    o, eo = silu(z, 0.0)
    return h * o, e * o.abs() * 1.001 + (h.abs() + e) * eo + 2 * U * (h * o).abs(), h, e


def backward(x, ag, xg, param, dy, ab=None, xb=None, z=None, scale=8.0, h0=None, dlast=None):
    """Gradients {name: (value, bound)}; rows (L, B, D), states (B, D)."""
    g = gates(x, ag, xg, param, ab, xb, scale)
    start = x.new_zeros(x.shape[1:]) if h0 is None else h0
    h, eh = run(g, start)
    L = x.shape[0]
    prev, eprev = torch.cat([start[None], h[:-1]]), torch.cat([torch.zeros_like(start)[None], eh[:-1]])
    out = {}
    gy, egy = dy, torch.zeros_like(dy)
    if z is not None:
        o, ro = sigmoid(z, z.abs())
        gy, egy = dy * z * o, (dy * z * o).abs() * (ro + 2 * U)
        k = 1 + z * (1 - o)
        ek = z.abs() * (o * ro + U) + k.abs() * 2 * U
        d = dy * h * o * k
        out["dz"] = d, (dy * o * k).abs() * eh * 1.01 + (dy * h * o).abs() * ek + d.abs() * (ro + 5 * U)
    G, e, m = torch.zeros_like(start), torch.zeros_like(start), torch.zeros_like(start)
    Gs, es = [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        if t == L - 1:
            add = torch.zeros_like(start) if dlast is None else dlast
            G, m, e = gy[t] + add, gy[t].abs() + add.abs(), egy[t] + U * (gy[t].abs() + add.abs())
        else:
            a = g["a"][t + 1]
            e = a * e + a * m * g["ra"][t + 1] + egy[t]
            G, m = gy[t] + a * G, gy[t].abs() + a * m
            e = e + 3 * U * m
        Gs[t], es[t] = G, e + 6 * U * m
    G, eG = torch.stack(Gs), torch.stack(es)
    la = g["l"] * g["a"]
    one, two = la * prev, g["u"] * g["q"]
    s = one + two
    es_ = la.abs() * eprev + one.abs() * (g["rl"] + g["ra"] + 3 * U) + two.abs() * (g["ru"] + g["rq"] + 3 * U)
    E = G * s
    eE = eG * (s.abs() + es_) + G.abs() * es_ + 2 * U * E.abs()
    r1, er1 = 1 - g["r"], g["r"] * g["rr"] + U
    i1, ei1 = 1 - g["i"], g["i"] * g["ri"] + U
    out["da_gate"] = E * r1, eE * r1 + E.abs() * er1 + eE * er1 + 2 * U * E.abs()
    wi = g["w"] * g["i"]
    dx = G * wi
    out["dx"] = dx, eG * wi + dx.abs() * (g["rw"] + g["ri"] + 4 * U) + eG * wi * 1e-4
    dxg = dx * x * i1
    out["dx_gate"] = dxg, (out["dx"][1] * i1 + (dx.abs() + out["dx"][1]) * ei1) * x.abs() + 4 * U * dxg.abs()
    deep = (40 + L * x.shape[1] / 64 / 16) * U  # additions that a term of a sum over rows passes
    for name, (v, ev) in (("da_bias", out["da_gate"]), ("dx_bias", out["dx_gate"]), ("da_param", (E * g["ratio"], eE * g["ratio"]))):
        out[name] = v.sum((0, 1)), (ev + deep * (v.abs() + ev)).sum((0, 1)) + (12 * U * v.sum((0, 1)).abs() if name == "da_param" else 0)
    first = g["a"][0] * G[0]
    out["dinitial_state"] = first, g["a"][0] * eG[0] + first.abs() * (g["ra"][0] + U)
    return out
