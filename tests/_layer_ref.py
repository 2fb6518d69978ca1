"""The layer operators in 64 bits, from their definitions, one token after another on the CPU.

Every function also runs with ``mag=True``: the same formula with every term replaced by its absolute
value. The result bounds the sum of the magnitudes that an output adds up, so that rounding errors of an
fp32 evaluation are at most (operations on a term's way) * 2^-24 * magnitude.
"""

from __future__ import annotations

import torch

F64 = torch.float64


def _silu(x, mag):
    y = x * torch.sigmoid(x)
    return y.abs() if mag else y


def _silu_slope(x, mag):
    g = torch.sigmoid(x)
    return g * (1 + x.abs() * (1 - g)) if mag else g * (1 + x * (1 - g))


def wide(x, mag=False):
    """Inputs in 64 bits (their magnitudes with ``mag``); None stays None."""
    if x is None:
        return None
    x = x.detach().cpu().to(F64)
    return x.abs() if mag else x


def bounds(x, cu):
    """(first row, end) of every sequence on the flat token axis."""
    if cu is None:
        n, S = x.shape[:2]
        return [(i * S, (i + 1) * S) for i in range(n)]
    cu = cu.tolist()
    return list(zip(cu, cu[1:]))


# ---------------------------------------------------------------- convolution
def conv(x, weight, bias, initial, cu, silu, dout=None, dstate=None, mag=False):
    """{"out", "state"} and, with dout, the gradients."""
    D, W = weight.shape
    X, w, n = wide(x, mag).reshape(-1, D), wide(weight, mag), len(bounds(x, cu))
    true = {"x": wide(x).reshape(-1, D), "w": wide(weight)}
    b, tb = (torch.zeros(D, dtype=F64),) * 2 if bias is None else (wide(bias, mag), wide(bias))
    zero = torch.zeros(n, W - 1, D, dtype=F64)
    s0, ts0 = (zero, zero) if initial is None else (wide(initial, mag), wide(initial))
    ds = zero if dstate is None else wide(dstate, mag)
    out, state = torch.zeros_like(X), torch.zeros_like(zero)
    dx, dw, db, ds0 = torch.zeros_like(X), torch.zeros_like(w), torch.zeros(D, dtype=F64), torch.zeros_like(zero)
    for i, (lo, hi) in enumerate(bounds(x, cu)):
        e, te = torch.cat([s0[i], X[lo:hi]]), torch.cat([ts0[i], true["x"][lo:hi]])
        de = torch.zeros_like(e)
        de[hi - lo:] += ds[i]
        for t in range(hi - lo):
            pre = b + (w.t() * e[t:t + W]).sum(0)
            tpre = tb + (true["w"].t() * te[t:t + W]).sum(0)
            # of the activation: its largest slope (about 1.1) carries errors of pre
            out[lo + t] = (1.1 * pre if mag else _silu(pre, False)) if silu else pre
            if dout is not None:
                g = wide(dout, mag).reshape(-1, D)[lo + t]
                # the slope changes by at most 0.5 per unit of pre
                dp = g * ((_silu_slope(tpre, True) + 0.5 * pre) if mag else _silu_slope(tpre, False)) if silu else g
                de[t:t + W] += w.t() * dp
                dw += (dp * e[t:t + W]).t()
                db += dp
        state[i] = e[hi - lo:]
        ds0[i], dx[lo:hi] = de[:W - 1], de[W - 1:]
    r = {"out": out.reshape(x.shape), "state": state}
    if dout is not None:
        r.update(dx=dx.reshape(x.shape), dweight=dw, dbias=db, dinitial_state=ds0)
    return r


# ---------------------------------------------------------------- scan
def softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def scan(u, dt, a, b, c, d, z, dt_bias, initial, cu, sp, dout=None, dstate=None, mag=False):
    D, N = a.shape
    G = b.shape[-2]
    n, shape = len(bounds(u, cu)), u.shape
    raw = wide(dt).reshape(-1, D) + (0 if dt_bias is None else wide(dt_bias))
    step = softplus(raw) if sp else raw
    slope = torch.sigmoid(raw) if sp else torch.ones_like(raw)
    A = wide(a)
    decay_of = lambda t: torch.exp(step[t][:, None] * A)  # noqa: E731
    st, Aw = (step.abs(), A.abs()) if mag else (step, A)
    U = wide(u, mag).reshape(-1, D)
    spread = lambda x: wide(x, mag).reshape(-1, G, N).repeat_interleave(D // G, 1)  # noqa: E731
    B, C = spread(b), spread(c)
    skip = torch.zeros(D, dtype=F64) if d is None else wide(d, mag)
    Z = None if z is None else wide(z).reshape(-1, D)
    zero = torch.zeros(n, D, N, dtype=F64)
    s0 = zero if initial is None else wide(initial, mag)
    T = U.shape[0]
    H, P = torch.zeros(T, D, N, dtype=F64), torch.zeros(T, D, N, dtype=F64)
    state = s0.clone()
    for i, (lo, hi) in enumerate(bounds(u, cu)):
        h = s0[i]
        for t in range(lo, hi):
            P[t] = h
            h = decay_of(t) * h + (st[t] * U[t])[:, None] * B[t]
            H[t] = h
        state[i] = h
    y = (H * C).sum(-1) + skip * U
    r = {"out": (y if Z is None else y * _silu(Z, mag)).reshape(shape), "state": state}
    if dout is None:
        return r
    g_out = wide(dout, mag).reshape(-1, D)
    dy = g_out if Z is None else g_out * _silu(Z, mag)
    g_of, ds0 = torch.zeros(T, D, N, dtype=F64), torch.zeros_like(zero)
    X = torch.zeros(T, D, N, dtype=F64)
    dS = zero if dstate is None else wide(dstate, mag)
    for i, (lo, hi) in enumerate(bounds(u, cu)):
        g = dS[i]
        for t in range(hi - 1, lo - 1, -1):
            g = g + C[t] * dy[t][:, None]
            g_of[t] = g
            g = g * decay_of(t)
            X[t] = g * P[t]
        ds0[i] = g
    sgb = (g_of * B).sum(-1)
    ddt = (U * sgb + (X * Aw).sum(-1)) * slope
    fold = lambda x: x.reshape(T, G, D // G, N).sum(2).reshape(b.shape)  # noqa: E731
    r.update(du=(st * sgb + skip * dy).reshape(shape), ddt=ddt.reshape(shape), da=(X * st[..., None]).sum(0),
             db=fold(g_of * (st * U)[..., None]), dc=fold(H * dy[..., None]), dd=(dy * U).sum(0), ddt_bias=ddt.sum(0),
             dinitial_state=ds0)
    if Z is not None:
        r["dz"] = (g_out * y * _silu_slope(Z, mag)).reshape(shape)
    return r


# ---------------------------------------------------------------- norm
def norm(x, weight, bias, z, groups, eps, center, gate, silu, dout=None, mag=False):
    D = x.shape[-1]
    X, w = wide(x).reshape(-1, D), wide(weight)
    Z = None if z is None else wide(z).reshape(-1, D)
    split = lambda t: t.reshape(-1, groups, D // groups)  # noqa: E731
    join = lambda t: t.reshape(-1, D)  # noqa: E731
    b = torch.zeros(D, dtype=F64) if bias is None else wide(bias)
    v = split(X * _silu(Z, False) if Z is not None and gate == "before" else X)
    m = v.mean(-1, keepdim=True) if center else torch.zeros_like(v[..., :1])
    r = 1 / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + eps)
    hat = join((v - m) * r)
    if mag:
        # centring cancels: a centred value carries the errors of v and m; those of r scale hat
        ma = v.abs().mean(-1, keepdim=True) if center else m
        hat_m = join((v.abs() + 3 * ma) * r)
        hat_m = hat_m + join(split(hat).abs() * (split(hat).abs() * split(hat_m)).mean(-1, keepdim=True))
        X, w, b = X.abs(), w.abs(), b.abs()
    else:
        hat_m = hat
    p, tp = hat_m * w + b, hat * wide(weight) + (0 if bias is None else wide(bias))
    after = Z is not None and gate == "after"
    if after:
        out = p * _silu(Z, mag)
    elif silu:
        out = 1.1 * p if mag else _silu(p, False)
    else:
        out = p
    res = {"out": out.reshape(x.shape)}
    if dout is None:
        return res
    g = wide(dout, mag).reshape(-1, D)
    if after:
        dp = g * _silu(Z, mag)
    elif silu:
        dp = g * ((_silu_slope(tp, True) + 0.5 * p) if mag else _silu_slope(tp, False))
    else:
        dp = g
    res["dweight"], res["dbias"] = (dp * hat_m).sum(0), dp.sum(0)
    q = split(dp * w)
    hm = split(hat_m)
    if mag:
        dv = q + hm * (q * hm).mean(-1, keepdim=True) + (q.mean(-1, keepdim=True) if center else 0)
        dv = join(dv * r * 2)       # and the error of r itself
    else:
        dv = q - hm * (q * hm).mean(-1, keepdim=True) - (q.mean(-1, keepdim=True) if center else 0)
        dv = join(dv * r)
    res["dx"] = (dv * _silu(Z, mag) if Z is not None and gate == "before" else dv).reshape(x.shape)
    if Z is not None:
        dz = dv * X if gate == "before" else g * p
        res["dz"] = (dz * _silu_slope(Z, mag)).reshape(x.shape)
    return res


# ---------------------------------------------------------------- comparison
def check(got, ref, mag, ops, what=""):
    """Every element within half a step of its type of the reference, plus ops * 2^-24 of its magnitude (and, for
    values under the type's normal range, half a step there). Returns the largest error in parts of that."""
    worst = 0.0
    for name, r in ref.items():
        x = got.get(name)
        if x is None:
            continue
        assert x.shape == r.shape, (what, name, x.shape, r.shape)
        f = torch.finfo(x.dtype)
        tol = f.eps / 2 * r.abs() + ops * 2.0 ** -24 * (1 + f.eps) * mag[name] + f.tiny * f.eps
        err = (x.detach().cpu().to(F64) - r).abs() / tol
        # terms beyond the largest fp32 number (2^128) have no fp32 sum to compare with; a gate that scales such a
        # sum by as little as 2^-25 leaves its product above 2^100
        err = torch.where(mag[name] < 2.0 ** 100, err, torch.zeros_like(err))
        assert not torch.isnan(err).any(), (what, name, "NaN")
        if err.numel():
            worst = max(worst, float(err.max()))
            assert float(err.max()) <= 1, (what, name, float(err.max()), int(err.argmax()))
    return worst
