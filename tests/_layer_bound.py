"""The selective scan in 64 bits with a bound on what an fp32 evaluation may be off by, carried through the recurrence.

An error that entered at token s reaches token t through the decays between them, so old errors fade as old terms do.
With E = 2^-24 (half a step of fp32), first order, h's magnitude M (the recurrence with every term positive) and the
decay p = exp(v a), v the step and x = dt + dt_bias:

* x carries 1, v through softplus 5 more (its own error is at most 2.6e-7 = 4.4 E): v's relative error is k E with
  k = 5 + |x| sigmoid(x) / v, or 1 without softplus; v u carries k + 1, v u b k + 2.
* p's argument v a log2(e) carries k + 3. Where the time axis is cut, p stands for a product of chunk decays
  exp(a sum v), whose sum carries at most one rounding for each of its L terms: k + 3 + L, times |v a|; the
  exponential's last place counts 2 and the multiply-add 1: r = (k + 3 + L) |v a| + 3.
* e[t] = p e[t-1] + r E p M[t-1] + (k + 3) E |v u b|, and the same for the adjoint g backwards.
* a sum of N products carries N + 8 (any order; joins over lanes and waves), a gate z sigmoid(z) 8 + 2 |z| (the
  exponential's argument twice over, exponential, sum, reciprocal, two products), its slope 14 + 2 |z|.
* a sum over tokens carries the L of a chunk, and the R partial rows over 64 accumulators and their join.

All outputs are compared, element by element, with half a step of their type and this bound (and, for values below the
type's normal range, half a step there).
"""

from __future__ import annotations

import torch

from . import _layer_ref as R

E = 2.0 ** -24
SUMS = ("da", "dd", "ddt_bias")     # over tokens: worst-case errors add up there, values of both signs do not


def scan(u, dt, a, b, c, d, z, dt_bias, initial, cu, sp, dout, dstate, chunk):
    """(reference, bound): dicts of the forward outputs and the gradients. ``chunk``: at least the tokens of a chunk that
    is cut (of one that is not, no sum of steps is taken)."""
    ref = R.scan(u, dt, a, b, c, d, z, dt_bias, initial, cu, sp, dout, dstate)
    D, N = a.shape
    G = b.shape[-2]
    spans, shape = R.bounds(u, cu), u.shape
    n, L = len(spans), chunk
    W = R.wide
    A = W(a)
    x = W(dt).reshape(-1, D) + (0 if dt_bias is None else W(dt_bias))
    v = R.softplus(x) if sp else x
    slope = torch.sigmoid(x) if sp else torch.ones_like(x)
    k = 5 + x.abs() * slope / v.clamp(min=1e-300) if sp else torch.ones_like(x)
    v = v.abs()
    U, B, C = W(u, True).reshape(-1, D), *(W(t, True).reshape(-1, G, N).repeat_interleave(D // G, 1) for t in (b, c))
    T = U.shape[0]
    skip = torch.zeros(D, dtype=R.F64) if d is None else W(d, True)
    Z = torch.zeros(T, D, dtype=R.F64) if z is None else W(z, True).reshape(-1, D)
    gate = torch.ones_like(Z) if z is None else R._silu(W(z), True).reshape(-1, D)
    gk = torch.zeros_like(Z) if z is None else 8 + 2 * Z
    zero = torch.zeros(n, D, N, dtype=R.F64)
    s0 = zero if initial is None else W(initial, True)
    raw = x if not sp else R.softplus(x)
    P = [torch.exp(raw[t][:, None] * A) for t in range(T)]
    Rr = [((k[t] + 3 + L) * v[t])[:, None] * A.abs() + 3 for t in range(T)]
    add = [(v[t] * U[t])[:, None] * B[t] for t in range(T)]
    M, e, Mp, ep = (torch.zeros(T, D, N, dtype=R.F64) for _ in range(4))
    st = torch.zeros_like(zero)
    for i, (lo, hi) in enumerate(spans):
        m, err = s0[i], torch.zeros(D, N, dtype=R.F64)
        for t in range(lo, hi):
            Mp[t], ep[t] = m, err
            err = P[t] * err + Rr[t] * E * P[t] * m + (k[t][:, None] + 3) * E * add[t]
            m = P[t] * m + add[t]
            M[t], e[t] = m, err
        st[i] = err + 4 * E * m
    sum_n = (N + 8) * E
    y = (M * C).sum(-1) + skip * U
    ey = (e * C).sum(-1) + sum_n * y
    bound = {"out": (gate * (ey + gk * E * y)).reshape(shape), "state": st}
    if dout is None:
        return ref, bound
    do = W(dout, True).reshape(-1, D)
    dy = do * gate
    g, eg, X, eX = (torch.zeros(T, D, N, dtype=R.F64) for _ in range(4))
    dS = zero if dstate is None else W(dstate, True)
    ds0 = torch.zeros_like(zero)
    for i, (lo, hi) in enumerate(spans):
        m, err = dS[i], torch.zeros(D, N, dtype=R.F64)
        for t in range(hi - 1, lo - 1, -1):
            new = C[t] * dy[t][:, None]
            err = err + (gk[t][:, None] + 3) * E * new
            m = m + new
            g[t], eg[t] = m, err
            X[t] = m * P[t] * Mp[t]
            eX[t] = P[t] * (err * Mp[t] + m * ep[t]) + (Rr[t] + 2) * E * X[t]
            err, m = P[t] * err + Rr[t] * E * P[t] * m, P[t] * m
        ds0[i] = err + 4 * E * m
    s, es = (g * B).sum(-1), (eg * B).sum(-1)
    es = es + sum_n * s
    xa = (X * A.abs()).sum(-1)
    exa = (eX * A.abs()).sum(-1) + (N + 12) * E * xa
    sum_t = _sum_ops(T, n, L) * E
    ddt = slope * (U * s + xa)
    eddt = slope * (U * es + exa) + (14 + 3 * x.abs()) * E * ddt
    w, kw = v * U, k + 2
    fold = lambda q: q.reshape(T, G, D // G, N).sum(2).reshape(b.shape)  # noqa: E731
    sum_d = (10 + D / (16 * G)) * E
    vX = v[..., None] * X
    zm = torch.ones_like(Z) if z is None else R._silu_slope(W(z), True).reshape(-1, D)
    bound.update(
        du=(v * (es + (k + 2) * E * s) + skip * dy * (gk + 3) * E).reshape(shape), ddt=eddt.reshape(shape),
        da=(v[..., None] * eX + (k[..., None] + 1) * E * vX).sum(0) + sum_t * vX.sum(0),
        db=fold(w[..., None] * eg + (kw[..., None] * E + sum_d) * g * w[..., None]),
        dc=fold(dy[..., None] * e + ((gk[..., None] + 2) * E + sum_d) * M * dy[..., None]),
        dd=((gk + 2) * E * dy * U).sum(0) + sum_t * (dy * U).sum(0),
        ddt_bias=eddt.sum(0) + sum_t * ddt.sum(0), dinitial_state=ds0)
    if z is not None:
        bound["dz"] = (do * zm * (ey + (14 + 2 * Z) * E * y)).reshape(shape)
    return ref, bound


def _sum_ops(T, n, chunk):
    return chunk + (T // 16 + n + 1) / 64 + 24


def check_sum(total, terms, n, chunk, what=""):
    """A sum over tokens against the terms that were stored in fp32: each term half a step, and the sum's additions."""
    x = terms.detach().cpu().to(R.F64).reshape(-1, total.shape[0])
    lim = 1.01 * (_sum_ops(x.shape[0], n, chunk) + 2) * E * x.abs().sum(0) + torch.finfo(torch.float32).tiny
    err = (total.detach().cpu().to(R.F64) - x.sum(0)).abs() / lim
    assert float(err.max()) <= 1, (what, float(err.max()))


def check(got, ref, bound, names, what=""):
    """Every named output is there and every element of it within its bound. Returns the largest error in parts of that,
    and the largest median of bound to value over the outputs."""
    worst = blunt = 0.0
    for name in names:
        x, r = got[name], ref[name]
        assert x is not None and x.shape == r.shape and r.numel() > 0, (what, name)
        assert bool(torch.isfinite(r).all()), (what, name, "the reference")
        x = x.detach().cpu()
        assert bool(torch.isfinite(x).all()), (what, name, "not finite")
        f = torch.finfo(x.dtype)
        lim = bound[name] * 1.01 * (1 + f.eps)
        err = (x.to(R.F64) - r).abs() / (f.eps / 2 * r.abs() + lim + f.tiny * f.eps)
        worst, k = max(worst, float(err.max())), int(err.argmax())
        assert float(err.max()) <= 1, (what, name, float(err.max()), k)
        blunt = max(blunt, float((lim / r.abs().clamp(min=1e-300)).median()))
    return worst, blunt
