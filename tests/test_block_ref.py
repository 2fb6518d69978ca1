"""The 64-bit references of the gated linear recurrence and of the residual addition's norm are pinned (no GPU needed): their
gradients against differences and against automatic differentiation of the definition, the generator against its published
answers."""

import pytest
import torch

from . import _block_ref as R

F64 = torch.float64


def _inputs(seqs, D, z, gen):
    n = len(seqs)
    T = sum(seqs)
    g = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    x = dict(x=g(T, D), r=g(T, D), i=g(T, D), decay=g(D) - 3, r_bias=g(D), i_bias=g(D), z=g(T, D) if z else None, initial=g(n, D))
    cu = torch.tensor([0] + seqs).cumsum(0)
    return x, cu, g(T, D), g(n, D)


def _define(x, r, i, decay, r_bias, i_bias, z, initial, cu, rate):
    """The definition, differentiable."""
    out, state = [], []
    for k, (lo, hi) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
        h = initial[k]
        for t in range(lo, hi):
            a = torch.exp(-rate * torch.nn.functional.softplus(decay) * torch.sigmoid(r[t] + r_bias))
            h = a * h + torch.sqrt(1 - a * a) * torch.sigmoid(i[t] + i_bias) * x[t]
            out.append(h if z is None else h * torch.nn.functional.silu(z[t]))
        state.append(h)
    return torch.stack(out), torch.stack(state)


@pytest.mark.parametrize("seqs", [[5], [1, 0, 3], [2, 2]])
@pytest.mark.parametrize("z", [True, False])
def test_recurrence_reference(seqs, z):
    x, cu, dout, ds = _inputs(seqs, 3, z, torch.Generator().manual_seed(len(seqs)))
    leaves = {k: v.clone().requires_grad_() for k, v in x.items() if v is not None}
    out, state = _define(**{**x, **leaves}, cu=cu, rate=5.0)
    ref, bound = R.recur(**x, cu=cu, rate=5.0, dout=dout, dstate=ds)
    assert torch.allclose(ref["out"], out, rtol=1e-12, atol=1e-13) and torch.allclose(ref["state"], state, rtol=1e-12, atol=1e-13)
    loss = (out * dout).sum() + (state * ds).sum()
    grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    for k, g in grads.items():
        name = "dinitial_state" if k == "initial" else "d" + k
        assert torch.allclose(ref[name], g, rtol=1e-9, atol=1e-11), name
        # and one difference along a random direction
        way = torch.randn(g.shape, generator=torch.Generator().manual_seed(7), dtype=F64)
        ends = []
        for s in (1e-6, -1e-6):
            o, st = _define(**{**x, k: x[k] + s * way}, cu=cu, rate=5.0)
            ends.append((o * dout).sum() + (st * ds).sum())
        assert abs(float((ends[0] - ends[1]) / 2e-6 - (g * way).sum())) < 1e-6 * (1 + float((g * way).abs().sum()))
    assert all(torch.isfinite(b).all() and (b >= 0).all() for b in bound.values())


def test_recurrence_where_nothing_enters():
    """exp(l) = 1 (a closed gate): the state stays, and r and decay get no part."""
    x, cu, dout, ds = _inputs([4], 2, False, torch.Generator().manual_seed(0))
    x["r"] = torch.full_like(x["r"], -2000.0)
    ref, _ = R.recur(**x, cu=cu, rate=8.0, dout=dout, dstate=ds)
    assert torch.equal(ref["state"], x["initial"])
    for k in ("dx", "dr", "di", "ddecay", "dr_bias", "di_bias"):
        assert torch.equal(ref[k], torch.zeros_like(ref[k])), k


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0), (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator(counter, key, want):
    assert tuple(R.philox(counter, key)) == want


def test_share_dropped():
    """16 bits against a threshold: the share is that of the threshold, within five standard deviations."""
    keep = R.kept((1234567890123, -5), 64, 512, 6554)
    p, n = 6554 / 65536, keep.numel()
    assert abs(float((~keep).double().mean()) - p) < 5 * (p * (1 - p) / n) ** 0.5


@pytest.mark.parametrize("drop", [False, True])
def test_norm_reference(drop):
    g = torch.Generator().manual_seed(3)
    T, D = 4, 11
    x, res, dout, ds = (torch.randn(T, D, generator=g, dtype=F64) for _ in range(4))
    w = torch.randn(D, generator=g, dtype=F64)
    mask, f = (R.kept((3, 4), T, D, 20000), 65536 / (65536 - 20000)) if drop else (None, 1.0)
    lx, lr, lw = (t.clone().requires_grad_() for t in (x, res, w))
    v = (lx if mask is None else lx * mask * f) + lr
    out = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-3) * lw
    ref, _ = R.add_norm(x, w, res, 1e-3, mask, f)
    assert torch.allclose(ref["out"], out, rtol=1e-12, atol=1e-13) and torch.allclose(ref["sum"], v, rtol=1e-12, atol=1e-13)
    dx, dr, dw = torch.autograd.grad((out * dout).sum() + (v * ds).sum(), (lx, lr, lw))
    got, _ = R.add_norm_grads(dout, v.detach(), w, ds, 1e-3, mask, f)
    for k, t in (("dx", dx), ("dresidual", dr), ("dweight", dw)):
        assert torch.allclose(got[k], t, rtol=1e-10, atol=1e-12), k
