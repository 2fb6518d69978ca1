"""The gated linear recurrence on the GPU at the ends of its parameters' range, with tokens far apart, and with what its forward
pass and its special values must not mix: stale workspaces, calls at once, sequences of a packed batch."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from . import _block_ref as R
from .test_gpu_block import _recur_inputs, _reference
from .test_gpu_layer import _gen, _need_gpu, _rows, _same  # noqa: F401

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32


def _params(x, decay, r_bias=None):
    x["decay"] = torch.tensor(decay, device="cuda")
    if r_bias is not None:
        x["r_bias"] = torch.tensor(r_bias, device="cuda")
    return x


# ---------------------------------------------------------------- decays near the smallest number
@pytest.mark.parametrize("S", [20, 200])
@pytest.mark.parametrize("rate,decay", [(0.05, [-86.9, -87.0, -87.3, -85.0, -84.0, -80.0, 0.0]), (2.0 ** -127, [-3.0, 0.0, 5.0, 100.0, 1e10, -20.0, 1e30]),
                                        (2.0 ** -149, [0.0, 3.0, 1e4, 1e20, 1e36, 1.0, -5.0]), (0.0, [0.0, -50.0, 20.0, 1e30, -100.0, 1.0, 3.0])])
def test_recur_of_the_smallest_rates(rate, decay, S):
    """rate softplus(decay) around 2^-126 and below it: nothing is forgotten or enters, and all gradients are finite and within the
    reference's bound."""
    g = _gen(S)
    D = len(decay)
    x = _params(_recur_inputs(g, (2, S), 2, D, FF), decay)
    dout, ds = _rows(g, (2, S), D, FF, False), torch.randn(2, D, generator=g).cuda()
    o = m.mamba_recur_fwd(**x, rate=rate, return_state=True)
    gr = m.mamba_recur_bwd(dout, **x, dstate=ds, rate=rate)
    for k, t in {**gr._asdict(), "out": o.out, "state": o.state}.items():
        assert torch.isfinite(t).all(), k
    ref, bound = _reference(x, None, rate, dout, ds)
    R.check({**gr._asdict(), "out": o.out, "state": o.state}, ref, bound, (rate, decay))


@pytest.mark.parametrize("S", [24, 200])
@pytest.mark.parametrize("dtype", [FF, BF])
def test_recur_of_steps_below_the_smallest_number(dtype, S):
    """A decay at the edge of fp32's range, or gates so shut, that 1 - exp(2 l) is below it while l is not yet zero: what it gives the
    gradients of r and decay is the limit's, not l over some constant."""
    g = _gen(S + 1)
    decay = [-87.0, -87.0, -87.0, -87.0, -86.0, -80.0, -5.0, 0.0]
    x = _params(_recur_inputs(g, (2, S), 2, 8, dtype), decay, [-3.0, -5.0, -9.0, 0.0, -6.0, -9.0, -86.0, -85.0])
    dout, ds = _rows(g, (2, S), 8, dtype, False), torch.randn(2, 8, generator=g).cuda()
    gr = m.mamba_recur_bwd(dout, **x, dstate=ds)
    ref, bound = _reference(x, None, 8.0, dout, ds)
    R.check(gr._asdict(), ref, bound, (dtype, S))


@pytest.mark.parametrize("size", [1e9, 1e12, 1e30, 3e38])
@pytest.mark.parametrize("S", [8, 150])
def test_recur_forgets_states_of_any_size(size, S):
    """Where a token keeps nothing (exp(l) = 0), a state of any size in front of it has no part in the gradients."""
    g = _gen(S + 2)
    decay = [3e38, 1e31, 1e30, 1e20, 1e6]
    x = _params(_recur_inputs(g, (2, S), 2, 5, FF), decay, [0.0] * 5)
    x["initial_state"] = size * x["initial_state"].sign()
    dout, ds = _rows(g, (2, S), 5, FF, False), torch.randn(2, 5, generator=g).cuda()
    o, gr = m.mamba_recur_fwd(**x, return_state=True), m.mamba_recur_bwd(dout, **x, dstate=ds)
    y = {**x, "initial_state": torch.zeros(2, 5, device="cuda")}
    p, gp = m.mamba_recur_fwd(**y, return_state=True), m.mamba_recur_bwd(dout, **y, dstate=ds)
    assert _same(o.out, p.out) and _same(o.state, p.state)
    for k, a, b in zip(gr._fields, gr, gp):
        assert torch.equal(a, b), k         # zeros may differ in sign
        assert torch.isfinite(a).all(), k
    for t in (gr.dr, gr.ddecay, gr.dr_bias, gr.dinitial_state):
        assert not t.any()


# ---------------------------------------------------------------- one token
@pytest.mark.parametrize("packed", [False, True])
def test_recur_with_one_token_whose_stride_is_far(packed):
    """One token of each sequence, in a buffer in which the next one would lie 2^26 elements and more behind it."""
    g = _gen(61)
    D, n = 40, 1 if packed else 4
    x = _recur_inputs(g, (n, 1), n, D, BF)
    dout = torch.randn(n, 1, D, generator=g).to(BF).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda") if packed else None
    near, far = {}, {}
    for k, t in {**x, "dout": dout}.items():
        if t.dim() == 3:
            near[k] = t[0] if packed else t
            far[k] = t.as_strided((1, D), ((1 << 26) + 8, 1)) if packed else t.as_strided((n, 1, D), (D, (1 << 26) + 8, 1))
        else:
            near[k] = far[k] = t
    a, b = (m.mamba_recur_fwd(**{k: v for k, v in y.items() if k != "dout"}, cu_seqlens=cu, return_state=True) for y in (near, far))
    assert _same(a.out, b.out) and _same(a.state, b.state)
    for p, q in zip(m.mamba_recur_bwd(**near, cu_seqlens=cu), m.mamba_recur_bwd(**far, cu_seqlens=cu)):
        assert _same(p, q)
