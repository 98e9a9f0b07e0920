"""The gated linear recurrence, layer norm and the backward passes from their
definitions, in 64 bits, with running bounds on what f32 arithmetic may be off by.

Bounds (u = 2^-24, an f32 rounding; |z| a gate's logit):
  sigmoid   relative S(z) = (|z| + 16) 4 u: its argument's rounding is |z| u in the
            exponent, the exponential and the reciprocal are good to 2^-22.
  decay     p = a r: S + 2 u.  e = exp(p): |p| (S + 10 u) + u where the series
            is taken (p > -1/4; 1 + s rounds once), 4 u elsewhere in place of the last u.
            m = sqrt(1 - e^2): half of what 1 - e is off by, relative, which is S + 12 u
            by the series and (e eps_e + u) / (1 - e) elsewhere, and 4 u.
  states    h_t = e h_{t-1} + b, b = m i x: with A the same on absolute values,
            E_t = e (E_{t-1} + (eps_e + 2 u) A_{t-1}) + (eps_b + 2 u) |b|; composing the
            pairs of rows instead rounds no more often.
  sums      of n terms by threads that hold at most n / 512 + 32 of them, and trees:
            (n / 512 + 64) u of the terms' sizes; a weight's gradient over the rows:
            (rows + 64) u.
The rest follows the formulas, each product adding its factors' relative errors
and a rounding.
"""
from __future__ import annotations

import math

import torch

from tests.mixer_ref import U, ranges, rounding  # noqa: F401


def _sig(z):
    return torch.sigmoid(z), (z.abs() + 16) * 4 * U


def _decay(a, r, eps_r):
    p = a * r
    e = torch.exp(p)
    less = -torch.expm1(p)
    small = p > -0.25
    eps_e = p.abs() * (eps_r + 10 * U) + torch.where(small, 1.0, 4.0) * U
    eps_less = torch.where(small, eps_r + 12 * U, (e * eps_e + U) / less.clamp(min=1e-300))
    m = torch.sqrt(-torch.expm1(2 * p))
    return p, e, eps_e, m, eps_less + 4 * U


def _start(i, state, slots, resume, width, step=False):
    """(slot or -1, the state that sequence i starts from)"""
    slot = -1
    if state is not None:
        slot = i if slots is None else int(slots[i])
        if not 0 <= slot < state.shape[0]:
            slot = -1
    go_on = slot >= 0 and (step or (resume is not None and bool(resume[i])))
    h = state[slot].double().cpu().clone() if go_on else torch.zeros(width, dtype=torch.float64)
    return slot, go_on, h


def recur(x, ig, rg, a, spans=None, state=None, slots=None, resume=None, step=False):
    """(out, bound, new state, its bound, state before each row, its bound) in f64; rows of
    no sequence are NaN."""
    x, ig, rg, a = (t.double().cpu() for t in (x, ig, rg, a))
    rows, width = x.shape
    i_, eps_i = _sig(ig)
    r_, eps_r = _sig(rg)
    _, e, eps_e, m, eps_m = _decay(a, r_, eps_r)
    b = m * i_ * x
    eps_b = eps_m + eps_i + 3 * U
    out = torch.full((rows, width), math.nan, dtype=torch.float64)
    bound, before, before_bound = (torch.full_like(out, math.nan) for _ in range(3))
    new = None if state is None else state.double().cpu().clone()
    new_bound = None if state is None else torch.zeros_like(new)
    for q, (r0, r1) in enumerate(spans):
        slot, _, h = _start(q, state, slots, resume, width, step)
        if step and slot < 0:
            continue
        A, E = h.abs(), torch.zeros_like(h)
        for t in range(r0, r1):
            before[t], before_bound[t] = h, E
            E = e[t] * (E + (eps_e[t] + 2 * U) * A) + (eps_b[t] + 2 * U) * b[t].abs()
            h = e[t] * h + b[t]
            A = e[t] * A + b[t].abs()
            out[t], bound[t] = h, E
        if slot >= 0:
            new[slot], new_bound[slot] = h, E
    return out, bound, new, new_bound, before, before_bound


def recur_backward(dout, x, ig, rg, a, spans, state=None, slots=None, resume=None, dstate=None):
    """{name: (gradient, bound)}: dx, di, dr (zeros in rows of no sequence), da, dh."""
    _, _, _, _, before, eps_h = recur(x, ig, rg, a, spans, state, slots, resume)
    dout, x, ig, rg, a = (t.double().cpu() for t in (dout, x, ig, rg, a))
    rows, width = x.shape
    i_, eps_i = _sig(ig)
    r_, eps_r = _sig(rg)
    _, e, eps_e, m, eps_m = _decay(a, r_, eps_r)
    over = torch.where(m > 0, r_ / m, torch.zeros_like(m))
    zero = torch.zeros(rows, width, dtype=torch.float64)
    got = {n: (zero.clone(), zero.clone()) for n in ("dx", "di", "dr")}
    dh, dh_bound = torch.zeros(len(spans), width, dtype=torch.float64), torch.zeros(
        len(spans), width, dtype=torch.float64)
    da, da_bound, da_size = (torch.zeros(width, dtype=torch.float64) for _ in range(3))
    for q, (r0, r1) in enumerate(spans):
        _, go_on, _ = _start(q, state, slots, resume, width)
        c = torch.zeros(width, dtype=torch.float64) if dstate is None else dstate[q].double().cpu()
        Ec, Ac = torch.zeros_like(c), c.abs()
        for t in range(r1 - 1, r0 - 1, -1):
            g, Ag = dout[t] + c, dout[t].abs() + Ac
            Eg = Ec + U * Ag
            dx = g * m[t] * i_[t]
            Edx = m[t] * i_[t] * Eg + dx.abs() * (eps_m[t] + eps_i[t] + 4 * U)
            less = 1 - i_[t]
            di = dx * x[t] * less
            Edi = (x[t] * less).abs() * Edx + (dx * x[t]).abs() * (eps_i[t] * i_[t] + U) + 4 * U * di.abs()
            t1, t2 = before[t] * e[t] * r_[t], i_[t] * x[t] * e[t] * e[t] * over[t]
            Et = (e[t] * r_[t] * eps_h[t] + t1.abs() * (eps_e[t] + eps_r[t] + 4 * U) +
                  t2.abs() * (eps_i[t] + 2 * eps_e[t] + eps_r[t] + eps_m[t] + 8 * U))
            size = t1.abs() + t2.abs()
            dpr = g * (t1 - t2)
            Edpr = g.abs() * Et + size * Eg + 2 * U * size * g.abs()
            less = 1 - r_[t]
            dr = a * dpr * less
            Edr = (a * less).abs() * Edpr + (a * dpr).abs() * (eps_r[t] * r_[t] + U) + 4 * U * dr.abs()
            for n, v, E in (("dx", dx, Edx), ("di", di, Edi), ("dr", dr, Edr)):
                got[n][0][t], got[n][1][t] = v, E
            da += dpr
            da_bound += Edpr
            da_size += dpr.abs()
            c, Ec = e[t] * g, e[t] * (Eg + (eps_e[t] + 2 * U) * Ag)
            Ac = e[t] * Ag
        if go_on:
            dh[q], dh_bound[q] = c, Ec + 2 * U * Ac
    got["da"] = (da, da_bound + (rows + 64) * U * da_size)
    got["dh"] = (dh, dh_bound)
    return got


def _sum_eps(n):
    return (n / 512 + 64) * U


def layer_norm(x, w, b, eps):
    """(out, bound) in f64."""
    x, w = x.double().cpu(), w.double().cpu()
    b = torch.zeros_like(w) if b is None else b.double().cpu()
    mean, d, Ed, n, En = _moments(x, eps)
    out = d * n * w + b
    return out, n * w.abs() * Ed + (d * n * w).abs() * (En + 3 * U) + 2 * U * out.abs()


def _moments(x, eps):
    """mean, d = x - mean, bound on d, n = 1 / sqrt(var + eps), relative bound on n"""
    s = _sum_eps(x.shape[1])
    mean = x.mean(1, keepdim=True)
    Em = (s + 2 * U) * x.abs().mean(1, keepdim=True)
    d = x - mean
    Ed = Em + U * d.abs()
    q = (d * d).mean(1, keepdim=True)
    Eq = 2 * (Ed * d.abs()).mean(1, keepdim=True) + (Ed * Ed).mean(1, keepdim=True) + (s + 3 * U) * q
    return mean, d, Ed, torch.rsqrt(q + eps), Eq / (2 * (q + eps)) + 4 * U


def layer_norm_backward(dout, x, w, eps):
    g, x, w = (t.double().cpu() for t in (dout, x, w))
    rows, width = x.shape
    s = _sum_eps(width)
    _, d, Ed, n, En = _moments(x, eps)
    u = g * w
    mu, mud = u.mean(1, keepdim=True), (u * d).mean(1, keepdim=True)
    Emu = (s + 3 * U) * u.abs().mean(1, keepdim=True)
    Emud = (u.abs() * Ed).mean(1, keepdim=True) + (s + 4 * U) * (u * d).abs().mean(1, keepdim=True)
    dx = n * (u - mu - d * n * n * mud)
    t2 = (d * n * n * mud).abs()
    Edx = (n * (Emu + d.abs() * n * n * Emud + n * n * mud.abs() * Ed) + n * t2 * 3 * En +
           n * (u - mu).abs() * En + 8 * U * n * (u.abs() + mu.abs() + t2))
    xh = d * n
    dw, db = (g * xh).sum(0), g.sum(0)
    Edw = (g.abs() * (n * Ed + xh.abs() * (En + 3 * U))).sum(0) + (rows + 64) * U * (g * xh).abs().sum(0)
    return {"dx": (dx, Edx), "dw": (dw, Edw), "db": (db, (rows + 64) * U * g.abs().sum(0))}


def norm_backward(dout, y, z, w, group, eps, mode):
    g, y, z, w = (t.double().cpu() for t in (dout, y, z, w))
    rows, width = y.shape
    s = _sum_eps(group)
    sig, eps_s = _sig(z)
    act, eps_a = z * sig, eps_s + U
    slope = sig * (1 + z * (1 - sig))
    Eslope = (sig * eps_s * (1 + z.abs() * (1 - sig)) + sig * z.abs() * (sig * eps_s + U) +
              4 * U * sig * (1 + z.abs() * (1 - sig)))

    def mean(t):
        return t.unflatten(1, (-1, group)).mean(2, keepdim=True).expand(
            rows, width // group, group).reshape(rows, width)

    wc = w.reshape(-1)
    wc = (wc if mode == "mamba2" else wc.repeat(width // group)).expand(rows, width)
    if mode == "mamba2":
        v, ev, u, eu = y * act, eps_a + U, g * wc, torch.full_like(g, 2 * U)
    else:
        v, ev, u, eu = y, torch.zeros_like(y), g * wc * act, eps_a + 3 * U
    q = mean(v * v)
    n = torch.rsqrt(q + eps)
    En = mean(v * v * (2 * ev + s + 3 * U)) / (2 * (q + eps)) + 4 * U
    uv = mean(u * v)
    Euv = mean((u * v).abs() * (ev + eu + s + 4 * U))
    k = n * n * uv
    dv = n * (u - v * k)
    size = n * (u.abs() + (v * k).abs())
    Edv = (n * (u.abs() * eu + v.abs() * n * n * Euv + (v * k).abs() * (ev + 2 * En + 4 * U)) +
           size * (En + 4 * U))
    if mode == "mamba2":
        dy, Edy = dv * act, act.abs() * Edv + (dv * act).abs() * (eps_a + 2 * U)
        dz = dv * y * slope
        Edz = (y * slope).abs() * Edv + (dv * y).abs() * Eslope + 3 * U * dz.abs()
        term, Eterm = g * v * n, (g * v * n).abs() * (ev + En + 4 * U)
    else:
        dy, Edy = dv, Edv
        dz = g * wc * y * n * slope
        Edz = (g * wc * y * n).abs() * (Eslope + (En + 5 * U) * slope.abs())
        term, Eterm = g * act * y * n, (g * act * y * n).abs() * (eps_a + En + 5 * U)
    terms = rows
    if mode == "onnx":
        term, Eterm = (t.reshape(-1, group) for t in (term, Eterm))
        terms = rows * (width // group)
    dw = term.sum(0)
    Edw = Eterm.sum(0) + (terms + 64) * U * term.abs().sum(0)
    return {"dy": (dy, Edy), "dgate": (dz, Edz), "dw": (dw, Edw)}


def assert_close(got, want, bound, dtype, what=""):
    """``got`` within the bound and its own rounding (which may also take the value over a
    midpoint: the factor) where ``want`` is a number."""
    got = got.double().cpu()
    tol = bound + (rounding(want, dtype) if dtype != torch.float32 else U * want.abs()) * (
        1 + 2.0 ** -8) + 1e-37
    fine = ~torch.isnan(want)
    worst = ((got - want).abs() - tol)[fine]
    assert worst.numel() == 0 or bool((worst <= 0).all()), (what, float(worst.max()))
    return fine
