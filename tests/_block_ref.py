"""The gated linear recurrence and the residual addition with its norm in 64 bits on the CPU, from their definitions, each
with a bound on the error of an evaluation in fp32.

Bounds count in units of u = 2^-24, the largest relative error of one fp32 rounding; hardware functions (2^x, reciprocal,
square root) are off by one step, 2 u. They are carried along with the values: a product's bound is that of either factor
times the other, a sum's the sum, each with its own rounding on top; "mag" values are the same formula with every term
replaced by its absolute value.

* sigmoid(q), q = p + bias: q has a rounding, -q log2(e) another, together 2 |q| u in the exponent, which reach the result
  times 1 - sigmoid; 2^x, the sum and the reciprocal are 5 u: 2 |q| (1 - s) + 6.
* l = -rate softplus(decay) s: softplus is within 2.6e-7 (5 u), three products: 10 more.
* a = 2^l2: |l| times the bound of l, and 2 for the function.
* 1 - a^2: as a series in l that bound and 6; elsewhere 2 a^2 / (1 - a^2) times that of a, where 2 a^2 |l| / (1 - a^2) <= 1 and
  4 a^2 / (1 - a^2) <= 15 for 2 |l| > 1/4: that of l and 20. Its root (or inverse root): half of it and 2.
* below 2^-126 the hardware's 2^x gives zero, and a product may: an absolute error of 2^-126 = 2^-102 u of a, of a g and of a x,
  which reaches what they are multiplied by (a g l h: with l = 300 it is far above the result's own smallest step). So may
  softplus (decay below -87): 2 l is off by up to f = 2 (rate + 1) 2^-126 more, and e = sqrt(1 - a^2) by sqrt(e^2 + f) - e, at most
  the lesser of sqrt(f) (4e-19 for a rate of 8) and f / e. l / e is e / 2 for small l, so it is off by no more.
* a state: each token multiplies its bound by a, adds the bounds of a and of what enters, and at most four roundings of
  the state's magnitude (folded, joined and walked again).
"""

from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24
FLUSH = 2.0 ** -102     # 2^-126, the smallest normal number, in u


def wide(x):
    return None if x is None else x.detach().cpu().to(F64)


def bounds_of(x, cu):
    """(first row, end) of every sequence on the flat token axis."""
    if cu is None:
        n, S = x.shape[:2]
        return [(i * S, (i + 1) * S) for i in range(n)]
    cu = cu.tolist()
    return list(zip(cu, cu[1:]))


def softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _sigmoid(p, bias):
    """(value, relative bound) for p + bias."""
    q, most = p + bias, p.abs() + bias.abs()
    s = torch.sigmoid(q)
    return s, 2 * most * (1 - s) + 6


def recur(x, r, i, decay, r_bias, i_bias, z, initial, cu, rate, dout=None, dstate=None):
    """({name: value}, {name: bound in u}) of the outputs and, with dout, the gradients."""
    shape, D, seqs = x.shape, x.shape[-1], bounds_of(x, cu)
    n = len(seqs)
    zero = torch.zeros(D, dtype=F64)
    flat = lambda v: wide(v).reshape(-1, D)  # noqa: E731
    X, Z = flat(x), None if z is None else flat(z)
    rb, ib = (zero if b is None else wide(b) for b in (r_bias, i_bias))
    (sr, csr), (si, csi) = _sigmoid(flat(r), rb), _sigmoid(flat(i), ib)
    sp = softplus(wide(decay))
    ell, cl = -rate * sp * sr, csr + 10
    a, e2 = torch.exp(ell), -torch.expm1(2 * ell)
    e, ca, ce = torch.sqrt(e2), ell.abs() * cl + 2, (cl + 20) / 2 + 2
    gone = 2 * (rate + 1) * 2.0 ** -126
    efl = torch.minimum(gone / e, torch.full_like(e, gone ** 0.5)) / U
    inv = torch.where(e > 0, 1 / e, torch.zeros_like(e))
    u = si * X
    b, cb = e * u, ce + csi + 2
    if Z is not None:
        sz, csz = _sigmoid(Z, zero)
        gate, cgate = Z * sz, csz + 2
    T = X.shape[0]
    s0 = torch.zeros(n, D, dtype=F64) if initial is None else wide(initial)
    prev, prev_m, prev_e, now, now_e = (torch.zeros(T, D, dtype=F64) for _ in range(5))
    now_m = torch.zeros(T, D, dtype=F64)
    state, state_e = s0.clone(), torch.zeros_like(s0)
    for k, (lo, hi) in enumerate(seqs):
        h, m, err = s0[k], s0[k].abs(), torch.zeros(D, dtype=F64)
        for t in range(lo, hi):
            prev[t], prev_m[t], prev_e[t] = h, m, err
            h = a[t] * h + b[t]
            err = a[t] * err + m * (a[t] * (ca[t] + 2) + FLUSH) + b[t].abs() * cb[t] + u[t].abs() * efl[t]
            m = a[t] * m + b[t].abs()
            err = err + 4 * m
            now[t], now_m[t], now_e[t] = h, m, err
        state[k], state_e[k] = h, err
    out = {"out": now if Z is None else now * gate, "state": state}
    bnd = {"out": now_e if Z is None else now_e * gate.abs() + now_m * gate.abs() * (cgate + 2), "state": state_e}
    if dout is not None:
        go = flat(dout)
        dh, dh_e = (go, torch.zeros_like(go)) if Z is None else (go * gate, (go * gate).abs() * (cgate + 2))
        G, Gm, Ge = (torch.zeros(T, D, dtype=F64) for _ in range(3))
        ds = torch.zeros(n, D, dtype=F64) if dstate is None else wide(dstate)
        d0, d0_e = ds.clone(), torch.zeros_like(ds)
        for k, (lo, hi) in enumerate(seqs):
            c, m, err = ds[k], ds[k].abs(), torch.zeros(D, dtype=F64)
            for t in range(hi - 1, lo - 1, -1):
                G[t], Gm[t] = dh[t] + c, dh[t].abs() + m
                Ge[t] = dh_e[t] + err + 2 * Gm[t]
                c, m = a[t] * G[t], a[t] * Gm[t]
                err = a[t] * Ge[t] + m * (ca[t] + 4) + FLUSH * Gm[t]
            d0[k], d0_e[k] = c, err
        la = ell.abs()
        t1, t2 = la * a * Gm * prev_m, la * inv * a * a * Gm * u.abs()
        W = a * G * (ell * prev - ell * inv * a * u)
        We = t1 * (ca + cl + 6) + a * la * (Ge * prev_m + Gm * prev_e) + t2 * (2 * ca + cl + ce + csi + 8) + la * inv * a * a * u.abs() * Ge
        We = We + 2 * FLUSH * la * (Gm + 1) * (prev_m + inv * u.abs() + 1) + Gm * (prev_m * gone / U + u.abs() * efl)
        Wm = t1 + t2
        dr, dr_e = (1 - sr) * W, (1 - sr) * (We + 2 * Wm) + Wm * (sr * (csr + 4) + 1)     # 1 + l / (rate softplus): four more roundings
        du = G * e
        # sums over the tokens: a wave's eight, eight waves, a sixteenth of the chunks in four sums, sixteen of those
        adds = 8 + 8 + T // 1024 + n + 20
        total = lambda v, err, m: (v.sum(0), (err + m * adds).sum(0))  # noqa: E731
        di, di_m = du * u * (1 - si), Gm * e * u.abs()
        lost = Gm * efl
        di_e = Ge * e * u.abs() * (1 - si) + di_m * ((1 - si) * (ce + csi + 5) + si * csi + 1) + lost * u.abs()
        ratio = torch.where(sp > 0, torch.sigmoid(wide(decay)) / sp, torch.ones_like(sp))
        dec, dec_e = total(W, We, Wm)
        out.update(dx=du * si, dr=dr, di=di, ddecay=ratio * dec, dinitial_state=d0)
        bnd.update(dx=Ge * e * si + Gm * e * si * (ce + csi + 3) + lost * si, dr=dr_e, di=di_e,
                   ddecay=ratio * (dec_e + Wm.sum(0) * (2 * wide(decay).abs() + 16)), dinitial_state=d0_e)
        out["dr_bias"], bnd["dr_bias"] = total(dr, dr_e, (1 - sr) * Wm)
        out["di_bias"], bnd["di_bias"] = total(di, di_e, di_m * (1 - si))
        if Z is not None:
            slope, slope_m = sz * (1 + Z * (1 - sz)), sz * (1 + Z.abs() * (1 - sz))
            slope_e = slope_m * (csz + 4) + sz * Z.abs() * (sz * csz + 1)
            y_e = a * prev_e + prev_m * (a * (ca + 2) + FLUSH) + b.abs() * (cb + 2) + u.abs() * efl + 2 * now_m
            out["dz"] = go * now * slope
            bnd["dz"] = go.abs() * (y_e * slope.abs() + now_m * (slope_e + 3 * slope_m))
    per_token = {"out", "dx", "dr", "di", "dz"}
    return ({k: v.reshape(shape) if k in per_token else v for k, v in out.items()},
            {k: v.reshape(shape) if k in per_token else v for k, v in bnd.items()})


# ---------------------------------------------------------------- residual addition and norm
def philox(counter, key):
    """Philox4x32 with ten rounds, in whole numbers: four words for a counter of four and a key of two."""
    c, (k0, k1) = list(counter), key
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k0, b & 0xffffffff, (a >> 32) ^ c[3] ^ k1, a & 0xffffffff]
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    return c


def kept(seed, rows, D, drop, chosen=None):
    """[rows, D] of truth values: which elements dropout leaves. ``chosen``: these rows alone."""
    s, o = (v & (2 ** 64 - 1) for v in seed)
    res = []
    for row in range(rows) if chosen is None else chosen:
        bits = []
        for c in range(-(-D // 8)):
            for w in philox((c, row, o & 0xffffffff, o >> 32), (s & 0xffffffff, s >> 32)):
                bits += [w & 0xffff, w >> 16]
        res.append([b >= drop for b in bits[:D]])
    return torch.tensor(res)


SUM_OPS = 16 + 6 + 16 + 4   # a thread's sixteen, six levels of lanes, sixteen waves, and the mean


def _norm_scale(v, verr, eps):
    """1 / sqrt(mean v^2 + eps) and its relative bound, from v with a bound."""
    q = (v * v).mean(-1, keepdim=True)
    err = q * SUM_OPS + (2 * v.abs() * verr).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(q + eps)
    return r, torch.where(q + eps > 0, err / (q + eps) / 2, torch.zeros_like(q)) + 5


def add_norm(x, weight, residual, eps, mask=None, factor=1.0):
    """({"sum", "out"}, bounds); mask [rows, D] of what dropout keeps."""
    D = x.shape[-1]
    X, w = wide(x).reshape(-1, D), wide(weight)
    if mask is not None:
        X = torch.where(mask, X * factor, torch.zeros_like(X))
    v, verr = X, X.abs() * (0 if mask is None else 2)
    if residual is not None:
        v = v + wide(residual).reshape(-1, D)
        verr = verr + v.abs()
    r, cr = _norm_scale(v, verr, eps)
    out = v * r * w
    res = {"sum": v, "out": out}
    bnd = {"sum": verr, "out": out.abs() * (cr + 3) + r * w.abs() * verr}
    return {k: t.reshape(x.shape) for k, t in res.items()}, {k: t.reshape(x.shape) for k, t in bnd.items()}


def scales(out, bound, block, top):
    """Scales of rows (block None) or of blocks of columns, their relative bound, and both spread over the columns."""
    D = out.shape[-1]
    o, e = out.reshape(-1, D), bound.reshape(-1, D)
    parts = list(zip(o.split(block or D, 1), e.split(block or D, 1)))
    s = torch.stack([p.abs().amax(-1).clamp(min=2.0 ** -100) / top for p, _ in parts], 1)
    c = torch.stack([(q.amax(-1) / p.abs().amax(-1).clamp(min=2.0 ** -100)) for p, q in parts], 1) + 4
    spread = lambda t: torch.cat([t[:, k:k + 1].expand(-1, p.shape[1]) for k, (p, _) in enumerate(parts)], 1)  # noqa: E731
    return s, c, spread(s), spread(c)


def add_norm_grads(dout, total, weight, dsum, eps, mask=None, factor=1.0):
    """({"dx", "dresidual", "dweight"}, bounds), from the sum as it is given."""
    D = dout.shape[-1]
    g, v, w = wide(dout).reshape(-1, D), wide(total).reshape(-1, D), wide(weight)
    rows = g.shape[0]
    r, cr = _norm_scale(v, torch.zeros_like(v), eps)
    hat, q = v * r, g * w
    m, mm = (q * hat).mean(-1, keepdim=True), (q * hat).abs().mean(-1, keepdim=True)
    me = mm * (SUM_OPS + cr + 4)
    dv = r * (q - hat * m)
    err = r * ((q.abs() + hat.abs() * mm) * (cr + 5) + hat.abs() * me)
    if dsum is not None:
        dv = dv + wide(dsum).reshape(-1, D)
        err = err + dv.abs()
    dx, dxe = dv, err
    if mask is not None:
        dx, dxe = (torch.where(mask, t * factor, torch.zeros_like(t)) for t in (dv, err + 2 * dv.abs()))
    res = {"dx": dx, "dresidual": dv, "dweight": (g * hat).sum(0)}
    bnd = {"dx": dxe, "dresidual": err, "dweight": ((g * hat).abs() * (cr + 2 + rows // 256 + 40)).sum(0)}
    fit = lambda k, t: t if k == "dweight" else t.reshape(dout.shape)  # noqa: E731
    return {k: fit(k, t) for k, t in res.items()}, {k: fit(k, t) for k, t in bnd.items()}


# ---------------------------------------------------------------- comparison
def check(got, ref, bound, what=""):
    """Every element within half a step of its type of the reference and the bound. Returns the largest error in parts of that."""
    worst = 0.0
    for name, r in ref.items():
        x = got.get(name)
        if x is None:
            continue
        assert x.shape == r.shape, (what, name, x.shape, r.shape)
        f = torch.finfo(x.dtype)
        tol = f.eps / 2 * r.abs() + U * (1 + f.eps) * bound[name] + f.tiny * f.eps + 2.0 ** -126
        err = (x.detach().cpu().to(F64) - r).abs() / tol
        assert not torch.isnan(err).any(), (what, name, "NaN")
        if err.numel():
            worst = max(worst, float(err.max()))
            assert float(err.max()) <= 1, (what, name, float(err.max()), int(err.argmax()))
    return worst
