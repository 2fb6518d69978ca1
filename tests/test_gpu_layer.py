"""The layer operators on the GPU against the 64-bit reference (tests/_layer_ref.py).

Tolerance, for every element: half a step of the output's type (the one rounding when it is stored) plus
ops * 2^-24 times the magnitude of the terms it adds up. ``ops`` counts the fp32 operations on the longest way of a
term:
* convolution: W multiply-adds and the bias twice over (forward of the gradient, then the taps), the exponential,
  reciprocal and products of SiLU and its slope (12, hardware functions at 1 ulp); for the filter's gradient the sum
  over the tokens of a chunk (at most 64) and over the partial sums in four accumulators;
* scan: a term passes at most S decays, each an exponential whose argument carries the errors of dt (softplus: 6) and of
  the product, times |dt a| exp(dt a) <= 0.37: 8 a token in all (where dt < 0 lets the state grow, |dt a| is not bounded
  so: the exponential's argument then carries three roundings, 3 |dt a| a token more); N multiply-adds of <c, h>, 40 for the functions; the
  gradients pass two recurrences and sum over D channels or S tokens;
* norm: the sum over a thread's 32 elements and eight levels of lanes and waves, three times (mean, variance, gradient).
"""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from . import _layer_ref as R
from ._parity import log

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mamba_mimo_chunked_amd import _lib
    _lib.lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(g, lead, D, dtype, strided, scale=1.0):
    """[*lead, D] on the GPU: dense, or a slice of wider rows that starts inside one."""
    x = torch.randn(*lead, 2 * D + 3 if strided else D, generator=g) * scale
    x = x.to(dtype).cuda()
    return x[..., 1:D + 1] if strided else x


def _lead(seqs):
    """(leading shape, cu_seqlens on the CPU, tokens): (B, S), or ("packed", lengths, tokens behind the last)."""
    if seqs[0] != "packed":
        return seqs, None, seqs[0]
    cu = [0]
    for x in seqs[1]:
        cu.append(cu[-1] + x)
    return (cu[-1] + seqs[2],), torch.tensor(cu, dtype=torch.int32), len(seqs[1])


def _cut(x, cu, inner):
    """A packed tensor without the tokens behind the last sequence."""
    return x if x is None or cu is None else x[:int(cu[-1])]


def _same(x, y):
    """Bit for bit, NaN among them."""
    if x is None or y is None:
        return x is y
    kind = torch.int32 if x.element_size() == 4 else torch.int16
    return x.dtype == y.dtype and torch.equal(x.contiguous().view(kind), y.contiguous().view(kind))


def _tail_is(x, cu, value):
    if cu is not None and x is not None:
        tail = x[int(cu[-1]):].float()
        assert torch.equal(tail, torch.full_like(tail, value))


PACKED = ("packed", [0, 1, 5, 0, 70, 33, 2], 9)

# ---------------------------------------------------------------- convolution
CONV = [  # dtype, taps, D, sequences, bias, initial state, silu, strided
    (BF, 4, 64, (2, 33), True, True, True, False), (HF, 4, 40, (1, 130), True, False, True, False), (FF, 4, 24, (3, 17), False, True, True, False),
    (BF, 4, 61, (2, 20), True, True, True, True), (BF, 3, 16, (1, 1), True, True, False, False), (FF, 2, 5, (4, 2), True, True, True, False),
    (BF, 4, 8, (2, 3), False, False, True, False), (HF, 2, 72, (1, 65), True, True, True, False), (FF, 3, 600, PACKED, True, True, True, False),
    (BF, 4, 264, PACKED, True, True, True, False), (HF, 4, 33, PACKED, True, False, False, True), (FF, 5, 20, (2, 50), True, True, True, False),
    (BF, 6, 44, (1, 40), True, True, True, False), (HF, 7, 12, PACKED, False, True, True, False), (BF, 8, 36, (2, 29), True, True, True, False),
    (FF, 8, 7, ("packed", [3, 0, 0, 9], 0), True, True, True, False), (BF, 4, 2056, (1, 300), True, True, True, False),
    (FF, 4, 4, ("packed", [200] + [1] * 70, 40), True, True, True, False), (BF, 3, 10, ("packed", [0, 0], 5), True, True, True, False),
    # around the backward pass's chunks: whole unrolled steps in packed sequences, equal chunks in dense ones
    (FF, 3, 9, ("packed", [13, 14, 15, 28, 1], 1), True, True, True, False), (HF, 8, 6, ("packed", [16, 17, 18, 34], 0), True, True, True, False),
    (BF, 4, 64, (1, 25), True, True, True, False), (FF, 5, 33, (2, 24), True, True, True, False), (BF, 2, 16, (3, 23), True, True, True, False),
]


@pytest.mark.parametrize("dtype,W,D,seqs,has_bias,has_init,silu,strided", CONV)
def test_conv(dtype, W, D, seqs, has_bias, has_init, silu, strided):
    log(f"[conv] {dtype} W={W} D={D} {seqs}")
    g = _gen(W * 1000 + D)
    lead, cu, n = _lead(seqs)
    act = "silu" if silu else None
    x, dout = _rows(g, lead, D, dtype, strided), _rows(g, lead, D, dtype, strided)
    w = (torch.randn(D, W, generator=g) / W ** 0.5).cuda()
    b = torch.randn(D, generator=g).cuda() if has_bias else None
    s0 = torch.randn(n, W - 1, D, generator=g).to(dtype).cuda() if has_init else None
    ds = torch.randn(n, W - 1, D, generator=g).to(dtype).cuda()
    cud = None if cu is None else cu.cuda()
    o = m.mamba_conv_fwd(x, w, b, s0, cud, activation=act, return_state=True)
    gr = m.mamba_conv_bwd(dout, x, w, b, s0, ds, cud, activation=act)
    torch.cuda.synchronize()
    ref, mag = (R.conv(_cut(x, cu, 1), w, b, s0, cu, silu, _cut(dout, cu, 1), ds, mag=k) for k in (False, True))
    got = {"out": _cut(o.out, cu, 1), "state": o.state, "dx": _cut(gr.dx, cu, 1), "dweight": gr.dweight, "dbias": gr.dbias, "dinitial_state": gr.dinitial_state}
    assert (gr.dbias is None) == (b is None) and (gr.dinitial_state is None) == (s0 is None)
    T = lead[0] if cu is not None else lead[0] * lead[1]
    log(f"  worst {R.check(got, ref, mag, 2 * W + 2 + 12 + 64 + T // 256, (dtype, W, D, seqs)):.3f}")
    assert torch.equal(o.state.cpu().double(), ref["state"])
    _tail_is(o.out, cu, 0.0)
    _tail_is(gr.dx, cu, 0.0)
    # a caller's output: written in place, rows behind the last sequence left as they were
    out = torch.full((*lead, D), 7.0, dtype=dtype, device="cuda")
    r = m.mamba_conv_fwd(x, w, b, s0, cud, activation=act, out=out)
    assert r.out is out and r.state is None
    assert _same(_cut(out, cu, 1), _cut(o.out, cu, 1))
    _tail_is(out, cu, 7.0)


STEP_IDX = [None, [2, 0, 5], [4, -1, 4, 9, 4, 1], [3] * 5, list(range(69, -1, -1)), [(k * 7) % 64 for k in range(140)]]


def _serial(idx, n, slots):
    """(row, slot) in the order they have to appear to be taken."""
    return [(i, i if idx is None else idx[i]) for i in range(n) if idx is None or 0 <= idx[i] < slots]


@pytest.mark.parametrize("idx", STEP_IDX)
@pytest.mark.parametrize("dtype,W,D,pad", [(BF, 4, 72, 0), (FF, 3, 21, 1), (HF, 8, 300, 5)])
def test_conv_step(dtype, W, D, pad, idx):
    g = _gen(D)
    n = 3 if idx is None else len(idx)
    slots = 70
    pool = torch.randn(slots, W - 1 + pad, D, generator=g).to(dtype).cuda()
    state, before = pool[:, :W - 1], pool.clone()
    x = _rows(g, (n,), D, dtype, bool(pad))
    w, b = (torch.randn(D, W, generator=g) / W ** 0.5).cuda(), torch.randn(D, generator=g).cuda()
    ind = None if idx is None else torch.tensor(idx, dtype=torch.int32).cuda()
    out = m.mamba_conv_step(x, state, w, b, ind, activation="silu")
    torch.cuda.synchronize()
    want, after = torch.zeros(n, D, dtype=torch.float64), before.cpu().double()
    mag = torch.zeros_like(want)
    for i, k in _serial(idx, n, slots):
        args = (x[i:i + 1, None], w, b, after[k:k + 1, :W - 1].clone(), None, True)
        r, rm = R.conv(*args), R.conv(*args, mag=True)
        want[i], mag[i] = r["out"][0, 0], rm["out"][0, 0]
        after[k, :W - 1] = r["state"][0]
    R.check({"out": out}, {"out": want}, {"out": mag}, W + 14, idx)
    assert torch.equal(pool.cpu().double(), after)


# ---------------------------------------------------------------- scan
def _scan_inputs(g, lead, n, D, G, N, dtype, sp=True, skip=True, gate=True, bias=True, init=True, strided=False):
    x = dict(u=_rows(g, lead, D, dtype, strided), dt=_rows(g, lead, D, dtype, strided, 0.5))
    if not sp:
        x["dt"] = x["dt"].abs() * 0.1
    x["a"] = -(torch.rand(D, N, generator=g) * 4 + 0.05).cuda()
    x["b"], x["c"] = (torch.randn(*lead, G, N, generator=g).to(dtype).cuda() for _ in range(2))
    if strided:
        x["b"] = torch.cat([x["b"], x["b"]], -2)[..., :G, :]
    x["d"] = torch.randn(D, generator=g).cuda() if skip else None
    x["z"] = _rows(g, lead, D, dtype, strided) if gate else None
    x["dt_bias"] = (torch.randn(D, generator=g) - 2).cuda() if bias else None
    x["initial_state"] = torch.randn(n, D, N, generator=g).cuda() if init else None
    return x


SCAN = [  # dtype, D, G, N, sequences, options
    (BF, 64, 1, 16, (1, 40), {}), (FF, 70, 1, 16, (2, 19), {}), (HF, 128, 2, 16, (2, 33), {}), (BF, 8, 1, 4, (1, 1), {}),
    (FF, 3, 1, 1, (3, 2), {}), (BF, 24, 3, 5, (1, 17), dict(sp=False)), (FF, 66, 2, 8, (1, 300), {}), (BF, 80, 1, 13, (2, 130), dict(gate=False)),
    (FF, 40, 2, 17, (1, 130), dict(skip=False)), (HF, 36, 1, 24, (2, 70), dict(bias=False)), (BF, 65, 1, 32, (1, 100), dict(strided=True)),
    (FF, 20, 4, 48, (1, 90), dict(init=False)), (BF, 48, 2, 64, (1, 150), {}), (HF, 33, 1, 64, (2, 16), dict(strided=True)),
    (FF, 18, 1, 100, (1, 80), {}), (BF, 40, 1, 128, (1, 100), {}), (FF, 72, 1, 16, ("packed", [0, 1, 5, 0, 170, 33, 2], 9), {}),
    (BF, 130, 2, 16, ("packed", [300, 0, 1, 129], 50), {}), (HF, 12, 1, 7, ("packed", [1], 0), dict(sp=False, gate=False, skip=False, bias=False, init=False)),
    (FF, 36, 2, 33, PACKED, dict(gate=False, init=False)), (BF, 68, 1, 3, PACKED, dict(strided=True)), (FF, 5, 1, 6, ("packed", [0, 0, 3], 0), {}),
    (FF, 64, 1, 16, ("packed", [2] * 65, 3), {}), (BF, 16, 16, 8, (2, 35), {}), (FF, 260, 1, 9, (1, 66), {}),
    (BF, 20, 1, 16, ("packed", [0, 0], 70), {}), (FF, 64, 1, 16, (40, 20), {}), (HF, 512, 1, 16, (70, 3), {}),
    # enough tiles that the states are split over few waves; a sequence much longer than the average of its batch
    (FF, 1024, 1024, 7, (2, 20), {}), (BF, 300, 300, 40, ("packed", [100, 3, 0, 70], 4), {}), (HF, 150, 150, 100, (1, 40), {}),
    (FF, 16, 1, 16, ("packed", [1] * 30 + [1500] + [0] * 5, 2), {}),
]


@pytest.mark.parametrize("dtype,D,G,N,seqs,opt", SCAN)
def test_scan(dtype, D, G, N, seqs, opt):
    log(f"[scan] {dtype} D={D} G={G} N={N} {seqs} {opt}")
    g = _gen(D * 100 + N)
    lead, cu, n = _lead(seqs)
    x = _scan_inputs(g, lead, n, D, G, N, dtype, **opt)
    sp = opt.get("sp", True)
    dout = _rows(g, lead, D, dtype, opt.get("strided", False))
    ds = torch.randn(n, D, N, generator=g).cuda()
    cud = None if cu is None else cu.cuda()
    o = m.mamba_scan_fwd(**x, cu_seqlens=cud, dt_softplus=sp, return_state=True)
    gr = m.mamba_scan_bwd(dout, **x, dstate=ds, cu_seqlens=cud, dt_softplus=sp)
    torch.cuda.synchronize()
    cut = {k: _cut(v, cu, 1) if k in ("u", "dt", "b", "c", "z") else v for k, v in x.items()}
    args = [cut[k] for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial_state")]
    ref, mag = (R.scan(*args, cu, sp, _cut(dout, cu, 1), ds, mag=k) for k in (False, True))
    S = max(b - a for a, b in R.bounds(cut["u"], cu))
    step = R.wide(cut["dt"]) + (0 if x["dt_bias"] is None else R.wide(x["dt_bias"]))
    grow = 0 if sp else 3 * max(0.0, -float(step.min())) * float(x["a"].abs().max())
    fwd = {"out": _cut(o.out, cu, 1), "state": o.state}
    log(f"  fwd worst {R.check(fwd, ref, mag, (8 + grow) * S + N + 40, ('fwd', D, N, seqs)):.3f}")
    got = {k: _cut(v, cu, 1) if k in ("du", "ddt", "db", "dc", "dz") else v for k, v in gr._asdict().items()}
    for k, src in (("dd", "d"), ("dz", "z"), ("ddt_bias", "dt_bias"), ("dinitial_state", "initial_state")):
        assert (got[k] is None) == (x[src] is None), k
    log(f"  bwd worst {R.check(got, ref, mag, 2 * (8 + grow) * S + N + D // G + 60, ('bwd', D, N, seqs)):.3f}")
    for t in (o.out, gr.du, gr.ddt, gr.db, gr.dc, gr.dz):
        _tail_is(t, cu, 0.0)
    out = torch.full((*lead, D), 7.0, dtype=dtype, device="cuda")
    m.mamba_scan_fwd(**x, cu_seqlens=cud, dt_softplus=sp, out=out)
    assert _same(_cut(out, cu, 1), _cut(o.out, cu, 1))
    _tail_is(out, cu, 7.0)


@pytest.mark.parametrize("idx", STEP_IDX)
@pytest.mark.parametrize("dtype,D,G,N,pad", [(BF, 64, 1, 16, 0), (FF, 21, 3, 5, 1), (HF, 40, 2, 64, 2), (FF, 300, 1, 1, 0), (BF, 12, 1, 128, 0),
                                             (FF, 6, 2, 30, 0), (BF, 70, 1, 8, 3), (FF, 9, 1, 100, 0)])
def test_scan_step(dtype, D, G, N, pad, idx):
    g = _gen(D + N)
    n, slots = 3 if idx is None else len(idx), 70
    pool = torch.randn(slots, D + pad, N, generator=g).cuda()
    state, before = pool[:, :D], pool.clone()
    x = _scan_inputs(g, (n,), n, D, G, N, dtype, strided=bool(pad), init=False)
    x.pop("initial_state")
    ind = None if idx is None else torch.tensor(idx, dtype=torch.int32).cuda()
    out = m.mamba_scan_step(**x, state=state, state_indices=ind, dt_softplus=True)
    torch.cuda.synchronize()
    want, after = torch.zeros(n, D, dtype=torch.float64), before.cpu().double()
    mag, smag = torch.zeros_like(want), after.abs()
    seen = {}
    for i, k in _serial(idx, n, slots):
        row = [x[q][i:i + 1, None] if q in ("u", "dt", "b", "c", "z") else x[q] for q in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
        r = R.scan(*row, after[k:k + 1, :D].clone(), None, True)
        rm = R.scan(*row, smag[k:k + 1, :D].clone(), None, True, mag=True)
        want[i], mag[i] = r["out"][0, 0], rm["out"][0, 0]
        after[k, :D], smag[k, :D] = r["state"][0], rm["state"][0]
        seen[k] = seen.get(k, 0) + 1
    ops = 8 * max(seen.values(), default=1) + N + 40
    R.check({"out": out, "state": pool}, {"out": want, "state": after}, {"out": mag, "state": smag}, ops, idx)
    idle = [k for k in range(slots) if k not in seen]
    assert torch.equal(pool[idle], before[idle]) and torch.equal(pool[:, D:], before[:, D:])


def test_optional_inputs_left_out():
    """No initial state, no gradient of the last state, nothing but the recurrence."""
    g = _gen(12)
    for S in (9, 16, 90, 400):
        x = _scan_inputs(g, (2, S), 2, 20, 2, 16, FF, sp=False, skip=False, gate=False, bias=False, init=False)
        dout = torch.randn(2, S, 20, generator=g).cuda()
        gr = m.mamba_scan_bwd(dout, **x)
        o = m.mamba_scan_fwd(**x)
        assert o.state is None and gr.dd is gr.dz is gr.ddt_bias is gr.dinitial_state is None
        args = [x[k] for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial_state")]
        ref, mag = (R.scan(*args, None, False, dout, None, mag=k) for k in (False, True))
        R.check({"out": o.out}, ref, mag, 8 * S + 56, S)
        R.check(gr._asdict(), ref, mag, 16 * S + 96, S)
        w = torch.randn(20, 3, generator=g).cuda()
        gc = m.mamba_conv_bwd(dout, x["u"], w)
        ref, mag = (R.conv(x["u"], w, None, None, None, False, dout, None, mag=k) for k in (False, True))
        assert gc.dbias is gc.dinitial_state is None
        R.check(gc._asdict(), ref, mag, 6 + 16 + 128, S)


def test_special_values():
    """a = -inf forgets at once, a = 0 and a step of zero keep everything, large steps and gates saturate; NaN in a
    parameter of one channel stays in that channel."""
    g = _gen(13)
    x = _scan_inputs(g, (1, 50), 1, 70, 1, 16, FF)
    x["a"][3] = float("-inf")
    x["a"][4] = 0.0
    x["dt"][0, :, 5] = -200.0
    x["dt"][0, :, 6] = 90.0
    x["z"][0, :, 7], x["z"][0, :, 8] = -300.0, 300.0
    args = [x[k].clone() for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial_state")]
    o = m.mamba_scan_fwd(**x, dt_softplus=True, return_state=True)
    ref, mag = (R.scan(*args, None, True, mag=k) for k in (False, True))
    R.check({"out": o.out, "state": o.state}, ref, mag, 8 * 50 + 56)
    y = m.mamba_scan_step(x["u"][:, 0], x["dt"][:, 0], x["initial_state"].clone(), x["a"],
                          x["b"][:, 0], x["c"][:, 0], x["d"], x["z"][:, 0], x["dt_bias"], dt_softplus=True)
    R.check({"out": y}, {"out": ref["out"][:, 0]}, {"out": mag["out"][:, 0]}, 64)
    x["a"][9, 2] = float("nan")
    p = m.mamba_scan_fwd(**x, dt_softplus=True, return_state=True)
    assert p.out[0, :, 9].isnan().all() and p.state[0, 9, 2].isnan()
    keep = [k for k in range(70) if k != 9]
    assert _same(p.out[..., keep], o.out[..., keep])


def test_far_offsets():
    """Tensors of more than 2^31 elements: what lies behind that gives what it gives alone."""
    T, D, n = (1 << 21) + 130, 1024, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = slice(T - n, T)
    u, z = (torch.empty(T, D, dtype=BF, device="cuda") for _ in range(2))
    for t in (u, z):
        t.normal_(generator=g)
    cu = torch.tensor([0, T - n, T], dtype=torch.int32).cuda()
    w = torch.randn(D, 4, generator=g, device="cuda")
    one = torch.tensor([0, n], dtype=torch.int32).cuda()
    c = m.mamba_conv_fwd(u, w, cu_seqlens=cu, activation="silu", return_state=True)
    c1 = m.mamba_conv_fwd(u[tail].clone(), w, cu_seqlens=one, activation="silu", return_state=True)
    assert _same(c.out[tail], c1.out) and _same(c.state[1], c1.state[0])
    gc, gc1 = m.mamba_conv_bwd(z, u, w, cu_seqlens=cu), m.mamba_conv_bwd(z[tail].clone(), u[tail].clone(), w, cu_seqlens=one)
    assert _same(gc.dx[tail], gc1.dx)
    y = m.mamba_norm_fwd(u, w[:, 0].contiguous(), None, z, groups=2)
    assert _same(y[tail], m.mamba_norm_fwd(u[tail].clone(), w[:, 0].contiguous(), None, z[tail].clone(), groups=2))
    gn = m.mamba_norm_bwd(z, u, w[:, 0].contiguous(), None, c.out, groups=2)
    gn1 = m.mamba_norm_bwd(z[tail].clone(), u[tail].clone(), w[:, 0].contiguous(), None, c.out[tail].clone(), groups=2)
    assert _same(gn.dx[tail], gn1.dx) and _same(gn.dz[tail], gn1.dz)
    del c, gc, y, gn
    a = -torch.rand(D, 16, generator=g, device="cuda") - 0.1
    b = torch.randn(T, 1, 16, generator=g, device="cuda").to(BF)
    bias = torch.full((D,), -2.0, device="cuda")
    s = m.mamba_scan_fwd(u, z, a, b, b, None, u, bias, None, cu, dt_softplus=True, return_state=True)
    ut, zt, bt = u[tail].clone(), z[tail].clone(), b[tail].clone()
    s1 = m.mamba_scan_fwd(ut, zt, a, bt, bt, None, ut, bias, None, one, dt_softplus=True, return_state=True)
    tol = dict(rtol=2 ** -7, atol=2 ** -7)      # other chunks: fp32 rounding, then at most a step of bf16 in values of about one
    assert torch.allclose(s.out[tail].float(), s1.out.float(), **tol) and torch.allclose(s.state[1], s1.state[0], rtol=1e-4, atol=1e-4)
    del s
    gs = m.mamba_scan_bwd(u, u, z, a, b, b, None, z, bias, None, None, cu, dt_softplus=True)
    g1 = m.mamba_scan_bwd(ut, ut, zt, a, bt, bt, None, zt, bias, None, None, one, dt_softplus=True)
    for k in ("du", "ddt", "dz"):
        p, q = getattr(gs, k)[tail].float(), getattr(g1, k).float()
        assert float((p - q).norm() / q.norm()) < 2 ** -8, k
    for k in ("db", "dc"):
        p, q = getattr(gs, k)[tail].float(), getattr(g1, k).float()
        assert float((p - q).norm() / q.norm()) < 2 ** -8, k
    # a pool whose last slot starts behind 2^31 elements
    del gs, u, z, b
    slots = (1 << 31) // (3 * D) + 3
    pool = torch.empty(slots, 3, D, dtype=BF, device="cuda")
    pool[-1].normal_(generator=g)
    alone, x = pool[-1:].clone(), ut[:1]
    y = m.mamba_conv_step(x, pool, w, None, torch.tensor([slots - 1], dtype=torch.int32).cuda())
    assert _same(y, m.mamba_conv_step(x, alone, w)) and _same(pool[-1], alone[0])
    del pool
    slots = (1 << 31) // (16 * D) + 3
    pool = torch.empty(slots, D, 16, device="cuda")
    pool[-1].normal_(generator=g)
    alone = pool[-1:].clone()
    y = m.mamba_scan_step(x, x, pool, a, bt[:1], bt[:1], state_indices=torch.tensor([slots - 1], dtype=torch.int32).cuda(), dt_softplus=True)
    assert _same(y, m.mamba_scan_step(x, x, alone, a, bt[:1], bt[:1], dt_softplus=True)) and _same(pool[-1], alone[0])


def test_scan_gradients_against_differences():
    """A central difference of the GPU forward pass in fp32 along random directions. With h = 2^-7 the truncation is h^2
    times third derivatives (about 1e-4 of the value), the rounding of an output sum 1e-6 / h."""
    g = _gen(11)
    x = _scan_inputs(g, (2, 75), 2, 40, 2, 16, FF)
    co, cs = torch.randn(2, 75, 40, generator=g).cuda(), torch.randn(2, 40, 16, generator=g).cuda()
    gr = m.mamba_scan_bwd(co, **x, dstate=cs, dt_softplus=True)
    names = dict(u="du", dt="ddt", a="da", b="db", c="dc", d="dd", z="dz", dt_bias="ddt_bias", initial_state="dinitial_state")

    def value(**kw):
        o = m.mamba_scan_fwd(**{**x, **kw}, dt_softplus=True, return_state=True)
        return float((o.out.double() * co).sum() + (o.state.double() * cs).sum())
    h = 2.0 ** -7
    for k, gk in names.items():
        v = torch.randn(x[k].shape, generator=g).cuda()
        if k == "a":
            v *= 0.1
        num = (value(**{k: x[k] + h * v}) - value(**{k: x[k] - h * v})) / (2 * h)
        ana = float((getattr(gr, gk).double() * v).sum())
        size = float((getattr(gr, gk).double() * v).square().sum().sqrt())
        assert abs(num - ana) <= 0.01 * size + 1e-3, (k, num, ana, size)


# ---------------------------------------------------------------- norm
NORM = [  # dtype, shape, groups, center, gate, silu, bias, strided
    (BF, (5, 64), 1, False, "before", False, False, False), (HF, (2, 3, 128), 2, True, "after", False, True, False),
    (FF, (7, 100), 5, False, None, False, True, False), (BF, (1, 1), 1, False, "before", False, True, False), (FF, (3, 2), 2, True, None, True, True, False),
    (BF, (37, 256), 1, True, "before", False, True, True), (HF, (9, 513), 1, False, "after", False, True, False), (FF, (4, 1040), 1, True, None, True, False, False),
    (BF, (6, 1000), 1, False, "before", False, False, False), (BF, (300, 16), 2, True, "before", False, True, False), (FF, (33, 24), 3, False, "after", False, True, False),
    (BF, (5, 2048), 1, False, "before", False, True, False), (HF, (3, 2049), 1, True, "before", False, True, False), (BF, (1030, 512), 2, False, "after", False, True, False),
    (BF, (3, 4096), 1, True, None, True, True, False), (FF, (2, 8192), 1, True, "before", False, True, False), (BF, (2, 8192), 1, False, "after", False, True, False),
    (HF, (2, 8191), 1, True, None, False, True, False), (FF, (70, 1500), 1, False, "before", False, True, True), (BF, (2, 16384), 2, True, "before", False, False, False),
    (FF, (2050, 7), 1, True, "after", False, True, False), (FF, (4, 400), 1, True, None, False, True, False), (BF, (8, 320), 1, False, None, True, True, False),
    (FF, (2, 4100), 1, False, "after", False, True, False), (BF, (64,), 1, False, None, False, False, False), (HF, (4, 300), 2, False, "before", False, True, False),
]


@pytest.mark.parametrize("dtype,shape,G,center,gate,silu,has_bias,strided", NORM)
def test_norm(dtype, shape, G, center, gate, silu, has_bias, strided):
    log(f"[norm] {dtype} {shape} G={G} {center} {gate} {silu}")
    D = shape[-1]
    g = _gen(D + G)
    x, dout = _rows(g, shape[:-1], D, dtype, strided), _rows(g, shape[:-1], D, dtype, strided)
    if center:
        x = (x.float() + 1.5).to(dtype)
    z = _rows(g, shape[:-1], D, dtype, strided) if gate else None
    w, b = torch.randn(D, generator=g).cuda(), torch.randn(D, generator=g).cuda() if has_bias else None
    kw = dict(groups=G, eps=1e-5, center=center, gate=gate or "before", activation="silu" if silu else None)
    out = m.mamba_norm_fwd(x, w, b, z, **kw)
    gr = m.mamba_norm_bwd(dout, x, w, b, z, **kw)
    torch.cuda.synchronize()
    ref, mag = (R.norm(x, w, b, z, G, 1e-5, center, gate or "before", silu, dout, mag=k) for k in (False, True))
    got = {"out": out, **gr._asdict()}
    assert (gr.dbias is None) == (b is None) and (gr.dz is None) == (z is None)
    rows = x.numel() // D
    log(f"  worst {R.check(got, ref, mag, 3 * 40 + 30 + rows // 64, (dtype, shape, G)):.3f}")
    res = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    assert m.mamba_norm_fwd(x, w, b, z, **kw, out=res) is res and _same(res, out)


# ---------------------------------------------------------------- together, and the manners of a call
class _Block:
    """Convolution, scan and norm in a row, as a layer uses them; prompt, gradient and single tokens."""

    def __init__(self, dtype, D=96, G=2, N=16, W=4, seed=21):
        g = _gen(seed)
        self.D, self.N, self.G, self.W, self.dtype = D, N, G, W, dtype
        C = D + 2 * G * N                       # the convolution runs over u, b and c
        self.cw, self.cb = (torch.randn(C, W, generator=g) / 2).cuda(), torch.randn(C, generator=g).cuda()
        self.a, self.d = -(torch.rand(D, N, generator=g) * 4 + 0.1).cuda(), torch.randn(D, generator=g).cuda()
        self.bias, self.nw = (torch.randn(D, generator=g) - 2).cuda(), torch.randn(D, generator=g).cuda()
        self.C = C

    def inputs(self, g, *lead):
        return tuple((torch.randn(*lead, k, generator=g) * 0.7).to(self.dtype).cuda() for k in (self.C, self.D, self.D))

    def split(self, xbc):
        D, GN = self.D, self.G * self.N
        return xbc[..., :D], xbc[..., D:D + GN].unflatten(-1, (self.G, self.N)), xbc[..., D + GN:].unflatten(-1, (self.G, self.N))

    def prompt(self, xbc, dt, z, cs=None, ss=None, cu=None):
        c = m.mamba_conv_fwd(xbc, self.cw, self.cb, cs, cu, activation="silu", return_state=True)
        u, b, cc = self.split(c.out)
        s = m.mamba_scan_fwd(u, dt, self.a, b, cc, self.d, None, self.bias, ss, cu, dt_softplus=True, return_state=True)
        return m.mamba_norm_fwd(s.out, self.nw, None, z, groups=self.G), c, s

    def step(self, xbc, dt, z, cs, ss, idx=None):
        u, b, c = self.split(m.mamba_conv_step(xbc, cs, self.cw, self.cb, idx, activation="silu"))
        y = m.mamba_scan_step(u, dt, ss, self.a, b, c, self.d, None, self.bias, idx, dt_softplus=True)
        return m.mamba_norm_fwd(y, self.nw, None, z, groups=self.G)

    def grads(self, dout, xbc, dt, z):
        _, c, s = self.prompt(xbc, dt, z)
        gn = m.mamba_norm_bwd(dout, s.out, self.nw, None, z, groups=self.G)
        u, b, cc = self.split(c.out)
        gs = m.mamba_scan_bwd(gn.dx, u, dt, self.a, b, cc, self.d, None, self.bias, dt_softplus=True)
        dxbc = torch.cat([gs.du, gs.db.flatten(-2), gs.dc.flatten(-2)], -1)
        gc = m.mamba_conv_bwd(dxbc, xbc, self.cw, self.cb, activation="silu")
        return [gc.dx, gc.dweight, gc.dbias, gs.ddt, gs.da, gs.dd, gs.ddt_bias, gn.dz, gn.dweight]


def test_prompt_then_steps_equals_a_longer_prompt():
    """In fp32: the states that a prompt leaves and the steps from them give what the longer prompt gives. Both sides
    are within the tolerances above of the same value; the norm divides by values of about one."""
    blk, g = _Block(FF), _gen(5)
    S, K, n = 150, 6, 3
    xbc, dt, z = blk.inputs(g, n, S + K)
    full, _, _ = blk.prompt(xbc, dt, z)
    _, c, s = blk.prompt(xbc[:, :S], dt[:, :S], z[:, :S])
    perm = torch.tensor([4, 0, 2], dtype=torch.int32).cuda()      # the states lie in a pool
    cs, ss = torch.zeros(5, *c.state.shape[1:], device="cuda"), torch.zeros(5, *s.state.shape[1:], device="cuda")
    cs[perm.long()], ss[perm.long()] = c.state, s.state
    for k in range(S, S + K):
        y = blk.step(xbc[:, k], dt[:, k], z[:, k], cs, ss, perm)
        assert torch.allclose(y, full[:, k], rtol=2e-4, atol=2e-4), k
    # and a second prompt that starts from the states of the first
    rest, _, _ = blk.prompt(xbc[:, S:], dt[:, S:], z[:, S:], c.state, s.state)
    assert torch.allclose(rest, full[:, S:], rtol=2e-4, atol=2e-4)


@pytest.mark.parametrize("dtype", [BF, FF])
def test_packed_equals_each_sequence_alone(dtype):
    """The chunk boundaries differ, so fp32 values agree to rounding: a step of the type, and the same for fp32 with
    the tolerance above."""
    blk, g = _Block(dtype), _gen(6)
    lens = [70, 1, 200, 33]
    xbc, dt, z = blk.inputs(g, sum(lens))
    cu = torch.tensor([0, 70, 71, 271, 304], dtype=torch.int32).cuda()
    y, c, s = blk.prompt(xbc, dt, z, cu=cu)
    tol = dict(rtol=2e-4, atol=2e-4) if dtype is FF else dict(rtol=2 ** -6, atol=2 ** -5)
    for i, (lo, hi) in enumerate(zip([0, 70, 71, 271], [70, 71, 271, 304])):
        y1, c1, s1 = blk.prompt(xbc[None, lo:hi], dt[None, lo:hi], z[None, lo:hi])
        assert torch.allclose(y[lo:hi].float(), y1[0].float(), **tol), i
        assert torch.equal(c.state[i], c1.state[0])
        assert torch.allclose(s.state[i], s1.state[0], rtol=1e-3, atol=1e-3 if dtype is FF else 2 ** -6), i


def test_equal_inputs_give_equal_bits():
    """Twice, and with a workspace that is full of NaN: no atomics, nothing read before it is written."""
    blk, g = _Block(BF), _gen(7)
    xbc, dt, z = blk.inputs(g, 2, 333)
    dout = torch.randn(2, 333, blk.D, generator=g).to(BF).cuda()
    one, two = blk.grads(dout, xbc, dt, z), blk.grads(dout, xbc, dt, z)
    for a, b in zip(one, two):
        assert _same(a, b)
    u, b, c = blk.split(xbc)
    args = (u, dt, blk.a, b, c, blk.d, z, blk.bias)
    ws = torch.full((1 << 26,), 255, dtype=torch.uint8, device="cuda")
    for x, y in zip(m.mamba_scan_bwd(dout, *args, dt_softplus=True), m.mamba_scan_bwd(dout, *args, dt_softplus=True, workspace=ws)):
        assert _same(x, y)
    ws.fill_(255)
    assert _same(m.mamba_scan_fwd(*args, dt_softplus=True).out, m.mamba_scan_fwd(*args, dt_softplus=True, workspace=ws).out)
    ws.fill_(255)
    for x, y in zip(m.mamba_conv_bwd(dout, u, blk.cw[:blk.D]), m.mamba_conv_bwd(dout, u, blk.cw[:blk.D], workspace=ws)):
        assert _same(x, y)
    ws.fill_(255)
    for x, y in zip(m.mamba_norm_bwd(dout, u, blk.nw, None, z), m.mamba_norm_bwd(dout, u, blk.nw, None, z, workspace=ws)):
        assert _same(x, y)


def test_captured_and_replayed():
    """Forward, backward and step in one graph, replayed with new inputs and eager work between the replays."""
    blk, g = _Block(BF), _gen(8)
    xbc, dt, z = blk.inputs(g, 2, 140)
    dout = torch.randn(2, 140, blk.D, generator=g).to(BF).cuda()
    sx, sd, sz = blk.inputs(g, 2)
    cs, ss = torch.randn(2, blk.W - 1, blk.C, generator=g).to(BF).cuda(), torch.randn(2, blk.D, blk.N, generator=g).cuda()
    idx = torch.tensor([1, 0], dtype=torch.int32).cuda()

    def all_of_it(cs, ss):
        return blk.grads(dout, xbc, dt, z) + [blk.prompt(xbc, dt, z)[0], blk.step(sx, sd, sz, cs, ss, idx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_of_it(cs.clone(), ss.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    gcs, gss = cs.clone(), ss.clone()
    with torch.cuda.graph(graph):
        got = all_of_it(gcs, gss)
    for k in range(4):
        for t in (xbc, dt, z, dout, sx, sd, sz):
            t.copy_((torch.randn(t.shape, generator=g) * 0.7).to(BF))
        gcs.copy_(cs)
        gss.copy_(ss)
        ecs, ess = cs.clone(), ss.clone()
        want = all_of_it(ecs, ess)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + [gcs, gss], want + [ecs, ess]):
            assert _same(a, b), k


def test_other_streams():
    """Two calls in flight on two streams, each with inputs made on it."""
    blk = _Block(FF)
    want, got, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    data = [blk.inputs(_gen(30 + k), 1, 400) for k in range(2)]
    for x in data:
        want.append(blk.prompt(*x)[0])
    torch.cuda.synchronize()
    for s, x in zip(streams, data):
        with torch.cuda.stream(s):
            got.append(blk.prompt(*[t.clone() for t in x])[0])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert _same(a, b)


def test_nothing_reaches_over_a_sequence():
    """NaN in one sequence, or behind the last, leaves the others as they were."""
    blk, g = _Block(BF), _gen(9)
    xbc, dt, z = blk.inputs(g, 120)
    cu = torch.tensor([0, 40, 41, 100], dtype=torch.int32).cuda()
    y, c, s = blk.prompt(xbc, dt, z, cu=cu)
    u, b, cc = blk.split(xbc)
    dout = torch.randn(120, blk.D, generator=g).to(BF).cuda()
    gr = m.mamba_scan_bwd(dout, u, dt, blk.a, b, cc, blk.d, z, blk.bias, cu_seqlens=cu, dt_softplus=True)
    for t in (xbc, dt, dout):
        t[100:] = float("nan")
    g2 = m.mamba_scan_bwd(dout, u, dt, blk.a, b, cc, blk.d, z, blk.bias, cu_seqlens=cu, dt_softplus=True)
    for p, q in zip(gr, g2):
        assert _same(p, q)
    for t in (xbc, dt):
        t[41:] = float("nan")
    y2, c2, s2 = blk.prompt(xbc, dt, z, cu=cu)
    assert torch.equal(y[:41], y2[:41]) and torch.equal(c.state[:2], c2.state[:2]) and torch.equal(s.state[:2], s2.state[:2])
    assert torch.isnan(y2[41:100].float()).any() and torch.equal(s2.state[2].isnan().any(), torch.tensor(True).cuda())
