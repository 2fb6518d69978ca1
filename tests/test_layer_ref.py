"""The 64-bit reference of the layer operators (tests/_layer_ref.py), on the CPU: its gradients against central
differences of its forward pass, along random directions of every input."""

import pytest
import torch

from . import _layer_ref as R

F64 = torch.float64


def _directional(fwd, leaves, grads, outs, gen):
    """sum over leaves of <grad, v> against the difference quotient of <outputs, cotangents> along v."""
    h = 1e-5
    for name, x in leaves.items():
        v = torch.randn(x.shape, generator=gen, dtype=F64)
        val = [sum((o * outs[k]).sum() for k, o in fwd(**{**leaves, name: x + s * h * v}).items() if k in outs) for s in (1, -1)]
        num = float(val[0] - val[1]) / (2 * h)
        ana = float((grads[name] * v).sum())
        # second-order error h^2 times third derivatives, and 64-bit cancellation 1e-16 / h
        assert abs(num - ana) <= 1e-7 * max(1.0, abs(ana), abs(float(val[0]))), (name, num, ana)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 9]])
def test_conv(silu, cu):
    g = torch.Generator().manual_seed(3)
    cu = None if cu is None else torch.tensor(cu)
    shape, n = ((9, 5), 3) if cu is not None else ((2, 6, 5), 2)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    leaves = dict(x=rnd(*shape), weight=rnd(5, 4), bias=rnd(5), initial=rnd(n, 3, 5))
    fwd = lambda x, weight, bias, initial: R.conv(x, weight, bias, initial, cu, silu)  # noqa: E731
    outs = {"out": rnd(*shape), "state": rnd(n, 3, 5)}
    r = R.conv(**leaves, cu=cu, silu=silu, dout=outs["out"], dstate=outs["state"])
    _directional(fwd, leaves, dict(x=r["dx"], weight=r["dweight"], bias=r["dbias"], initial=r["dinitial_state"]), outs, g)


@pytest.mark.parametrize("sp,gated", [(True, True), (False, False)])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 8]])
def test_scan(sp, gated, cu):
    g = torch.Generator().manual_seed(4)
    cu = None if cu is None else torch.tensor(cu)
    lead, n = ((8,), 3) if cu is not None else ((2, 5), 2)
    D, G, N = 6, 2, 3
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    leaves = dict(u=rnd(*lead, D), dt=rnd(*lead, D) if sp else rnd(*lead, D).abs() * 0.3, a=-torch.rand(D, N, generator=g, dtype=F64) - 0.1,
                  b=rnd(*lead, G, N), c=rnd(*lead, G, N), d=rnd(D), dt_bias=rnd(D), initial=rnd(n, D, N))
    if gated:
        leaves["z"] = rnd(*lead, D)
    fwd = lambda u, dt, a, b, c, d, dt_bias, initial, z=None: R.scan(u, dt, a, b, c, d, z, dt_bias, initial, cu, sp)  # noqa: E731
    outs = {"out": rnd(*lead, D), "state": rnd(n, D, N)}
    r = R.scan(**{"z": None, **leaves}, cu=cu, sp=sp, dout=outs["out"], dstate=outs["state"])
    names = dict(u="du", dt="ddt", a="da", b="db", c="dc", d="dd", dt_bias="ddt_bias", initial="dinitial_state", z="dz")
    _directional(fwd, leaves, {k: r[names[k]] for k in leaves}, outs, g)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate,silu", [("before", False), ("after", False), (None, False), (None, True)])
def test_norm(center, gate, silu):
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    leaves = dict(x=rnd(3, 12), weight=rnd(12), bias=rnd(12))
    if gate:
        leaves["z"] = rnd(3, 12)
    fwd = lambda x, weight, bias, z=None: R.norm(x, weight, bias, z, 3, 1e-3, center, gate or "before", silu)  # noqa: E731
    outs = {"out": rnd(3, 12)}
    r = R.norm(**{"z": None, **leaves}, groups=3, eps=1e-3, center=center, gate=gate or "before", silu=silu, dout=outs["out"])
    _directional(fwd, leaves, {k: r["d" + k] for k in leaves}, outs, g)
