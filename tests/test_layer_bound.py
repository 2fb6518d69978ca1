"""The scan's error bound (tests/_layer_bound.py) on the CPU: correctly rounded results are within it, and results with a
mistake planted in the 64-bit reference are not, in fp32 and for every length."""

import pytest
import torch

from . import _layer_bound as Bd
from . import _layer_ref as R

FF = torch.float32
GRADS = ("du", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dinitial_state")


def _inputs(lead, D, G, N, n, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = dict(u=r(*lead, D), dt=r(*lead, D) * 0.5, a=-(torch.rand(D, N, generator=g) * 4 + 0.05), b=r(*lead, G, N), c=r(*lead, G, N), d=r(D),
             z=r(*lead, D), dt_bias=r(D) - 2, initial=r(n, D, N))
    return x, r(*lead, D), r(n, D, N)


def _rounded(ref):
    return {k: v.to(FF) for k, v in ref.items()}


CASES = [((1, 1), 3, 1, 1, None), ((1, 60), 8, 2, 5, None), ((1600,), 4, 1, 16, [0, 20, 20, 1600])]


@pytest.mark.parametrize("lead,D,G,N,cu", CASES)
def test_rounded_results_pass(lead, D, G, N, cu):
    cu = None if cu is None else torch.tensor(cu)
    x, do, ds = _inputs(lead, D, G, N, 1 if cu is None else 3)
    ref, bound = Bd.scan(**x, cu=cu, sp=True, dout=do, dstate=ds, chunk=128)
    got = _rounded(ref)
    # a typical element of a token is pinned to a part in 1000 of its value, one of the sums over tokens to 5 %
    assert Bd.check(got, ref, bound, [k for k in ("out", "state") + GRADS if k not in Bd.SUMS])[1] < 1e-3
    assert Bd.check(got, ref, bound, Bd.SUMS)[1] < 0.05
    Bd.check_sum(got["ddt_bias"], got["ddt"], 3, 128)


# what a mistake changes: inputs of the reference, by name
MISTAKES = {
    "a step off by 2^-8 at one token": dict(dt=lambda t: t.index_add(-2, torch.tensor([700]), torch.full((1, t.shape[-1]), 2.0 ** -8))),
    "a decay off by a part in 500": dict(a=lambda t: t * 1.002),
    "one token's b left out": dict(b=lambda t: t.index_fill(-3, torch.tensor([700]), 0.0)),
    "the state lost between two chunks": dict(cu=lambda t: torch.tensor([0, 768, 1600])),
}


@pytest.mark.parametrize("what", MISTAKES)
def test_mistakes_are_found(what):
    """In a sequence of 1600 tokens, in the outputs and in the gradients alike; the larger ones in the sums over tokens too."""
    x, do, ds = _inputs((1600,), 4, 1, 16, 1)
    cu = torch.tensor([0, 1600])
    ref, bound = Bd.scan(**x, cu=cu, sp=True, dout=do, dstate=ds, chunk=128)
    kw = {**x, "cu": cu, "dout": do, "dstate": ds}
    kw.update({k: f(kw[k]) for k, f in MISTAKES[what].items()})
    if kw["cu"].numel() == 3:       # two sequences in place of one
        kw.update(initial=torch.cat([x["initial"], torch.zeros_like(x["initial"])]), dstate=torch.cat([torch.zeros_like(ds), ds]))
    bad = R.scan(**kw, sp=True)
    if bad["state"].shape != ref["state"].shape:
        bad["state"], bad["dinitial_state"] = bad["state"][1:], bad["dinitial_state"][:1]
    bad = _rounded(bad)
    for name in ("out", "ddt") + (("da", "ddt_bias") if what.startswith(("one", "the")) else ()):
        with pytest.raises(AssertionError):
            Bd.check(bad, ref, bound, (name,), what)
    part = bad["ddt"].double()[:-16].sum(0).to(FF)      # a sum that leaves out a unit
    with pytest.raises(AssertionError):
        Bd.check_sum(part, bad["ddt"], 1, 128)
