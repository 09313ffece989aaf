"""Plain 64-bit forms of the serving operators, one sequence and one step after another, each with a
bound on what fp32 arithmetic may be off by.

The bounds count roundings.  u = 2^-24 is the largest relative error of one fp32 rounding; a hardware
exp2, log2 or reciprocal is taken as 2 u (one unit in the last place).  Products and sums of
quantities with relative errors add those errors; a state's error runs through the recurrence with
the state itself.  A value stored in a type t is off by at most eps(t) / 2 of itself more."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TINY = 1e-36  # exp2 and products may flush subnormals


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().cpu().double()


def silu(v, ev):
    """(silu(v), its error bound) for v off by at most ev: |silu'| <= 1.1; the exponent v log2(e) is off by
    1.5 |v| u in a factor e^-v whose weight in the quotient is at most 1, the rest is four roundings."""
    s = v * torch.sigmoid(v)
    return s, 1.1 * ev + s.abs() * (6 + 3 * v.abs()) * U


def step_dt(delta, bias, softplus):
    """(dt, its relative error bound).  v = delta + bias is rounded once; softplus(v) moves by at most
    |v| u sigmoid / softplus <= |v| u for v <= 0 and by less for v > 0, the exponent's rounding adds
    1.5 |v| u, the logarithm's and the sum's roundings at most 6 u."""
    v = delta + (0.0 if bias is None else bias)
    if not softplus:
        return v, torch.full_like(v, U) if bias is not None else torch.zeros_like(v)
    # the sum's rounding is relative to the larger of its terms where they cancel
    mag = delta.abs() + (0.0 if bias is None else bias.abs())
    return torch.nn.functional.softplus(v, threshold=1e9), (8 + 3 * mag) * U


def scan_steps(x, delta, A, B, C, D, z, bias, softplus, h0):
    """One sequence: x (L, dim), B (L, N), h0 (dim, N) in 64 bits.  Returns y, its bound, h, its bound."""
    L = x.shape[0]
    dt, rdt = step_dt(delta, bias, softplus)
    h, m, e = h0.clone(), h0.abs(), torch.zeros_like(h0)
    ys, es = [], []
    for t in range(L):
        d, rd = dt[t][:, None], rdt[t][:, None]
        a = torch.exp(d * A)
        u = d * x[t][:, None] * B[t][None, :]
        # relative error of a: the exponent's (dt's, A log2(e)'s two roundings, the product's) times its size, exp2's
        ra = (rd + 3 * U) * (d * A).abs() + 2 * U
        ru = rd + 3 * U
        h_new = a * h + u
        m_new = a * m + u.abs()
        e = a * e + a * m * ra + u.abs() * ru + m_new * 1.01 * U
        # a state whose terms leave fp32's range has no fp32 value: no bound from there on
        e = torch.where(m_new < 2.0 ** 126, e, torch.inf)
        h, m = h_new, m_new
        n = A.shape[1]
        cm = (C[t].abs()[None, :] * m).sum(1)
        acc = (C[t][None, :] * h).sum(1)
        err = (C[t].abs()[None, :] * e).sum(1) + (n + 4) * U * cm
        err = torch.where((cm < 2.0 ** 126) & ~err.isnan(), err, torch.inf)
        if D is not None:
            acc = acc + D * x[t]
            err = err + 2 * U * (D * x[t]).abs()
        if z is not None:
            g, eg = silu(z[t], 0.0)
            err = err * g.abs() * 1.001 + acc.abs() * eg + 2 * U * (acc * g).abs()
            acc = acc * g
        ys.append(acc)
        es.append(err)
    if not L:
        return x.new_zeros(0, x.shape[1]), x.new_zeros(0, x.shape[1]), h, e
    return torch.stack(ys), torch.stack(es), h, e


def conv_rows(line, weight, bias, act):
    """line (W + L, dim): the window, then the inputs.  Returns y (L, dim) and its bound."""
    k = weight.shape[1]
    L = line.shape[0] - (k - 1)
    acc = torch.zeros(L, line.shape[1], dtype=torch.float64) + (0.0 if bias is None else bias)
    mag = acc.abs()
    for j in range(k):
        term = line[j:j + L] * weight[:, j]
        acc, mag = acc + term, mag + term.abs()
    err = (k + 1) * U * mag
    return silu(acc, err) if act else (acc, err)


def check(got, ref, err, dtype, what):
    """|got - ref| within the bound and half a step of the storage type, element by element."""
    g = f64(got)
    tol = err + (ref.abs() + err) * (half_step(dtype) if dtype != torch.float32 else U) + TINY
    tol = torch.where(torch.isnan(err), torch.inf, tol) if torch.isinf(err).any() else tol
    bad = ~((g - ref).abs() <= tol) & ~(torch.isnan(g) & torch.isnan(ref)) & ~torch.isinf(tol)
    if ref.numel():
        ratio = ((g - ref).abs() / tol).nan_to_num(0.0).max().item()
        print(f"  {what}: worst error {ratio:.3f} of its bound", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, first at {bad.nonzero()[0].tolist()}"


def quantise(v):
    """codes (int64) and scales (float32, as numpy) of rows (..., N) in numpy float32."""
    v = np.asarray(v, np.float32)
    top = np.abs(v).max(-1)
    with np.errstate(all="ignore"):
        scale = (top.astype(np.float64) / 127.0).astype(np.float32)
        scale = np.where(np.isfinite(top), scale, np.float32(np.nan))
        q = v.astype(np.float64) / np.where(scale > 0, scale, 1).astype(np.float64)[..., None]
    q = np.clip(np.rint(np.where(np.isfinite(scale)[..., None], q, 0.0)), -127, 127)
    return np.where((scale == 0)[..., None], 0, q).astype(np.int64), scale
