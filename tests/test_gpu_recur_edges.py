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


@pytest.mark.parametrize("S", [20, 150])
@pytest.mark.parametrize("rate", [0.0, 2.0 ** -149, 2.0 ** -130, 2.0 ** -100, 1.0])
def test_recur_of_the_largest_decays(rate, S):
    """rate softplus(decay) of the largest decays: nothing is forgotten with a rate of zero, and what a small rate leaves of them counts."""
    g = _gen(S + 3)
    decay = [3.4e38, 2.4e38, 2.3e38, 1e38, 1.0]
    x = _params(_recur_inputs(g, (2, S), 2, 5, FF), decay)
    dout, ds = _rows(g, (2, S), 5, FF, False), torch.randn(2, 5, generator=g).cuda()
    o, gr = m.mamba_recur_fwd(**x, rate=rate, return_state=True), m.mamba_recur_bwd(dout, **x, dstate=ds, rate=rate)
    got = {**gr._asdict(), "out": o.out, "state": o.state}
    for k, t in got.items():
        assert torch.isfinite(t).all(), k
    ref, bound = _reference(x, None, rate, dout, ds)
    R.check(got, ref, bound, rate)
    s = x["initial_state"].clone()
    one = {k: x[k][:, 0].contiguous() for k in "xriz"}
    y = m.mamba_recur_step(state=s, **one, decay=x["decay"], r_bias=x["r_bias"], i_bias=x["i_bias"], rate=rate)
    assert torch.isfinite(y).all() and _same(y, o.out[:, 0])


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


# ---------------------------------------------------------------- workspaces and calls at once
SEVERAL = [  # dtype, D, leading axes, ends of packed sequences: several chunks, several groups of them
    (BF, 130, (2, 500), None), (FF, 33, (1, 9000), None), (HF, 64, (3, 300), None), (BF, 72, (3000,), [0, 700, 700, 2900]), (FF, 20, (900,), [15 * k for k in range(61)]),
]


@pytest.mark.parametrize("dtype,D,lead,ends", SEVERAL)
def test_recur_forward_whatever_lies_in_the_workspace(dtype, D, lead, ends):
    """Words that look told, counters and a mark that are set, and what a call on other data left: equal bits all the same."""
    g = _gen(D)
    n = len(ends) - 1 if ends else lead[0]
    cu = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, other = (_recur_inputs(g, lead, n, D, dtype) for _ in range(2))
    want = m.mamba_recur_fwd(**x, cu_seqlens=cu, return_state=True)
    assert torch.isfinite(want.out).all()
    for byte in (0x3f, 0, 1, 255):
        ws = torch.full((1 << 23,), byte, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            got = m.mamba_recur_fwd(**x, cu_seqlens=cu, return_state=True, workspace=ws)
            assert _same(got.out, want.out) and _same(got.state, want.state), byte
            m.mamba_recur_fwd(**other, cu_seqlens=cu, workspace=ws)                      # the same places, other words
            y = {k: v[..., :1000, :] if k in ("x", "r", "i", "z") else v for k, v in other.items()} if ends is None else other
            m.mamba_recur_fwd(**y, cu_seqlens=None if cu is None else torch.tensor([0] * n + [lead[0]], dtype=torch.int32, device="cuda"), workspace=ws)


def test_recur_forward_on_two_streams_at_once():
    """Blocks of two calls that wait for blocks of their own call, each with its own workspace: the bits of calls one by one."""
    g = torch.Generator(device="cuda").manual_seed(62)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    calls = []
    for n, S, D in ((1, 16384, 2048), (2, 9000, 1000)):
        x = {k: new(n, S, D).to(BF) for k in ("x", "r", "i", "z")}
        x.update(decay=new(D) - 3, r_bias=new(D), i_bias=new(D), initial_state=new(n, D))
        calls.append((x, torch.full((1 << 23,), 0x3f, dtype=torch.uint8, device="cuda"), torch.empty_like(x["x"])))
    want = [m.mamba_recur_fwd(**x, return_state=True) for x, _, _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (x, ws, out), s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append([m.mamba_recur_fwd(**x, return_state=True, workspace=ws, out=out) for _ in range(3)])
        torch.cuda.synchronize()
        for q, ref in zip(got, want):
            assert all(_same(o.out, ref.out) and _same(o.state, ref.state) for o in q)


# ---------------------------------------------------------------- special values
LENGTHS = [300, 0, 200, 70, 129, 5, 64, 1]


def _packed(g, D, dtype):
    ends = [0]
    for k in LENGTHS:
        ends.append(ends[-1] + k)
    T = ends[-1] + 7
    x = _recur_inputs(g, (T,), len(LENGTHS), D, dtype)
    return x, _rows(g, (T,), D, dtype, False), torch.randn(len(LENGTHS), D, generator=g).cuda(), torch.tensor(ends, dtype=torch.int32, device="cuda"), ends


TOKEN_GRADS, PARAM_GRADS = ("dx", "dr", "di", "dz"), ("ddecay", "dr_bias", "di_bias")


@pytest.mark.parametrize("dtype", [FF, BF])
@pytest.mark.parametrize("seq,at", [(0, 0), (0, 130), (2, 199), (4, 64), (7, 0)])
def test_recur_special_values_in_a_packed_batch(dtype, seq, at):
    """NaN and infinities of a token stay in their sequence and channel, forward and backward, and reach no token that does not
    follow (an input) or precede (a gradient) it; its channel's parameters' gradients are NaN where it has a part in them."""
    D, c = 70, 33
    x, dout, ds, cu, ends = _packed(_gen(63), D, dtype)
    clean, grads = m.mamba_recur_fwd(**x, cu_seqlens=cu, return_state=True), m.mamba_recur_bwd(dout, **x, dstate=ds, cu_seqlens=cu)
    lo, hi, t = ends[seq], ends[seq + 1], ends[seq] + at
    nan, inf = float("nan"), float("inf")
    rows = torch.arange(x["x"].shape[0], device="cuda")[:, None]
    mine = (torch.arange(D, device="cuda") == c)[None]
    for name, value in (("x", nan), ("x", inf), ("x", -inf), ("r", nan), ("i", nan), ("z", nan), ("initial_state", nan), ("dout", nan), ("dout", inf), ("dstate", nan)):
        y = {k: v.clone() if k == name else v for k, v in {**x, "dout": dout, "dstate": ds}.items()}
        y[name][seq if name in ("initial_state", "dstate") else t, c] = value
        gr = m.mamba_recur_bwd(**y, cu_seqlens=cu)
        o = m.mamba_recur_fwd(**{k: y[k] for k in x}, cu_seqlens=cu, return_state=True)
        whole = mine & (rows >= lo) & (rows < hi)
        later, here, before = whole & (rows >= t), whole & (rows == t), whole & (rows <= t)
        none = whole & (rows < lo)
        hit_out = {"x": later, "r": later, "i": later, "z": here, "initial_state": whole}.get(name, none)
        hit = {"x": later, "i": later, "z": before, "initial_state": whole, "dout": before, "dstate": whole}.get(name, whole)
        assert _same(o.out[~hit_out], clean.out[~hit_out]), (name, value)
        assert not torch.isfinite(o.out[hit_out & (rows == t)]).any(), (name, value)
        others = torch.ones(len(LENGTHS), D, dtype=torch.bool, device="cuda")
        others[seq, c] = False
        assert _same(o.state[others], clean.state[others]), (name, value)
        for k in TOKEN_GRADS:
            assert _same(getattr(gr, k)[~hit], getattr(grads, k)[~hit]), (name, value, k)
        assert _same(gr.dinitial_state[others], grads.dinitial_state[others]), (name, value)
        for k in PARAM_GRADS:
            a, b = getattr(gr, k), getattr(grads, k)
            assert _same(a[~mine[0]], b[~mine[0]]), (name, value, k)
            # di has no part of the states
            if name in ("r", "dstate") or (name == "initial_state" and k != "di_bias") or (name == "dout" and value != value):
                assert not torch.isfinite(a[c]), (name, value, k)


# ---------------------------------------------------------------- cu_seqlens against the rules
def test_recur_forward_with_ends_that_decrease():
    """A chunk waits for one that nobody has: the wait ends by its limit, nothing outside the output is written, what lies in front
    of the wait is right, and the next call with the same workspace is."""
    g = _gen(64)
    D, S = 72, 600
    x = _recur_inputs(g, (S,), 3, D, FF)
    good = torch.tensor([0, 500, 500, 600], dtype=torch.int32, device="cuda")
    want = m.mamba_recur_fwd(**x, cu_seqlens=good, return_state=True)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    room = torch.full((S + 64, D), 7.0, device="cuda")
    # chunks of 64: sequence 0 has slots 0 to 7 and tells no end, sequence 2 takes the slots 8 to 10 for its chunks 5 to 7, which look
    # at slot 7; their tokens begin at 100 + 320
    bad = torch.tensor([0, 500, 100, 600], dtype=torch.int32, device="cuda")
    m.mamba_recur_fwd(**x, cu_seqlens=bad, out=room[32:-32], workspace=ws)
    torch.cuda.synchronize()
    edge = torch.full((32, D), 7.0, device="cuda")
    assert torch.equal(room[:32], edge) and torch.equal(room[-32:], edge)
    assert _same(room[32:32 + 420], want.out[:420])
    assert torch.isnan(room[32 + 500:-32]).all()
    again = m.mamba_recur_fwd(**x, cu_seqlens=good, return_state=True, workspace=ws)
    assert _same(again.out, want.out) and _same(again.state, want.state)
