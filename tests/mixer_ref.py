"""The mixer's convolution and scan from their definitions, in 64 bits and one
row at a time, with a running bound on what f32 arithmetic may be off by.

Bounds (u = 2^-24, an f32 rounding):
  conv  the sum of taps + 1 terms in any order: (taps + 2) u sum|terms|, through
        silu (slope at most 1.1); silu itself (|v| + 16) * 4 u relative: its
        argument's rounding is |v| u in the exponent, the base-2 exponential
        and the reciprocal are good to 2^-22.
  scan  S_t = e S_{t-1} + z.  e carries the errors of dt (softplus: 6 u
        relative; its inputs' sum: |v| u absolute, at most that relative by
        softplus' slope over its value, 1 + |v|) and of its exponential (2 u and
        the product's rounding |dt a| u), so its relative error is at most
        eps_dt |dt a| + (4 + |dt a|) u; an update rounds twice more.  With E the
        bound on S's error and A the same recurrence on absolute values,
        E_t = e (E_{t-1} + (eps_e + 2 u) A_{t-1}) + (eps_dt + 4 u) |z|,
        and y is off by at most E_t |C| + (N + 4) u A_t |C| + 4 u |d x|.
  A rounding to T is eps_T / 2 relative (plus half the smallest subnormal).
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def rounding(t: torch.Tensor, dtype) -> torch.Tensor:
    f = torch.finfo(dtype)
    return t.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def ranges(rows: int, cu=None, seqs: int = 1):
    if cu is None:
        each = rows // seqs
        return [(i * each, (i + 1) * each) for i in range(seqs)]
    return list(zip(cu[:-1], cu[1:]))


def conv(x, w, bias=None, act=True, spans=None, state=None, slots=None, resume=None, step=False):
    """(out, bound, new state) in f64; rows of no sequence are NaN in out.
    ``state``: [slots, taps - 1, width] or None."""
    x, w = x.double().cpu(), w.double().cpu()
    bias = torch.zeros(x.shape[1], dtype=torch.float64) if bias is None else bias.double().cpu()
    taps = w.shape[1]
    out = torch.full(x.shape, math.nan, dtype=torch.float64)
    bound = torch.zeros_like(out)
    new = None if state is None else state.cpu().clone()
    for i, (b, e) in enumerate(spans):
        slot = -1
        if state is not None:
            slot = i if slots is None else int(slots[i])
            if not 0 <= slot < state.shape[0]:
                slot = -1
        if step and slot < 0:
            continue
        go_on = slot >= 0 and (step or (resume is not None and bool(resume[i])))
        old = state[slot].double().cpu() if go_on else torch.zeros(taps - 1, x.shape[1],
                                                                   dtype=torch.float64)
        u = torch.cat([old, x[b:e]])
        for t in range(e - b):
            terms = u[t:t + taps].t() * w
            v = terms.sum(1) + bias
            size = (terms.abs().sum(1) + bias.abs()) * (taps + 2) * U
            if act:
                y = v / (1 + torch.exp(-v))
                bound[b + t] = 1.1 * size + y.abs() * (v.abs() + 16) * 4 * U
                out[b + t] = y
            else:
                out[b + t], bound[b + t] = v, size
        if slot >= 0:
            new[slot] = u[u.shape[0] - (taps - 1):].to(state.dtype)
    return out, bound, new


def scan(x, dt, a, b, c, head_dim, state_size, d=None, dt_bias=None, softplus=True,
         limits=(0.0, math.inf), spans=None, state=None, slots=None, resume=None, step=False):
    """(out, bound, A|C| of each row, new state, its bound, its A) in f64."""
    x, dt, b, c = (t.double().cpu() for t in (x, dt, b, c))
    a = a.double().cpu()
    rows, H, P, N = x.shape[0], a.numel(), head_dim, state_size
    G = b.shape[1] // N
    zero = torch.zeros(H, dtype=torch.float64)
    d = zero if d is None else d.double().cpu()
    dt_bias = zero if dt_bias is None else dt_bias.double().cpu()
    xs = x.reshape(rows, H, P)
    bs = b.reshape(rows, G, N).repeat_interleave(H // G, 1)
    cs = c.reshape(rows, G, N).repeat_interleave(H // G, 1)
    v = dt + dt_bias
    dts = torch.logaddexp(v, torch.zeros_like(v)) if softplus else v
    dts = torch.where(dts < limits[0], torch.full_like(dts, limits[0]), dts)
    dts = torch.where(dts > limits[1], torch.full_like(dts, limits[1]), dts)
    eps_dt = torch.where(torch.isfinite(v), (1 + v.abs() + 6) * U, torch.zeros_like(v))  # 0, inf: exact
    out = torch.full((rows, H, P), math.nan, dtype=torch.float64)
    bound, size = torch.zeros_like(out), torch.zeros_like(out)
    new = None if state is None else state.double().cpu().clone()
    new_bound = None if state is None else torch.zeros_like(new)
    new_size = None if state is None else torch.zeros_like(new)
    for i, (r0, r1) in enumerate(spans):
        slot = -1
        if state is not None:
            slot = i if slots is None else int(slots[i])
            if not 0 <= slot < state.shape[0]:
                slot = -1
        if step and slot < 0:
            continue
        go_on = slot >= 0 and (step or (resume is not None and bool(resume[i])))
        S = state[slot].double().cpu().clone() if go_on else torch.zeros(H, P, N,
                                                                         dtype=torch.float64)
        A, E = S.abs(), torch.zeros_like(S)
        for t in range(r0, r1):
            p = dts[t] * a
            e = torch.exp(p)[:, None, None]
            eps_e = (eps_dt[t] * p.abs() + (4 + p.abs()) * U)[:, None, None]
            z = (dts[t][:, None] * xs[t])[..., None] * bs[t][:, None]
            E = e * (E + (eps_e + 2 * U) * A) + (eps_dt[t][:, None, None] + 4 * U) * z.abs()
            S = e * S + z
            A = e * A + z.abs()
            ca = cs[t].abs()[:, None]
            out[t] = (S * cs[t][:, None]).sum(-1) + d[:, None] * xs[t]
            dx = (d[:, None] * xs[t]).abs()
            size[t] = (A * ca).sum(-1) + dx
            bound[t] = (E * ca).sum(-1) + (N + 4) * U * size[t] + 4 * U * dx
        if slot >= 0:
            new[slot], new_bound[slot], new_size[slot] = S, E + 2 * U * A, A
    flat = lambda t: t.reshape(rows, H * P)  # noqa: E731
    return flat(out), flat(bound), flat(size), new, new_bound, new_size
