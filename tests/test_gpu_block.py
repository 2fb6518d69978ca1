"""The gated linear recurrence and the residual addition with its norm on the GPU against the 64-bit reference
(tests/_block_ref.py), within half a step of an output's type and the bound that the reference carries along."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from . import _block_ref as R
from ._parity import log
from .test_gpu_layer import PACKED, STEP_IDX, _cut, _gen, _lead, _need_gpu, _rows, _same, _serial, _tail_is  # noqa: F401

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
E4, I8 = torch.float8_e4m3fn, torch.int8


# ---------------------------------------------------------------- gated linear recurrence
def _recur_inputs(g, lead, n, D, dtype, gate=True, bias=True, init=True, strided=False, slow=3.0):
    x = {k: _rows(g, lead, D, dtype, strided) for k in ("x", "r", "i")}
    x["decay"] = (torch.randn(D, generator=g) * 2 - slow).cuda()
    x["r_bias"], x["i_bias"] = (torch.randn(D, generator=g).cuda() if bias else None for _ in range(2))
    x["z"] = _rows(g, lead, D, dtype, strided) if gate else None
    x["initial_state"] = torch.randn(n, D, generator=g).cuda() if init else None
    return x


def _reference(x, cu, rate, dout=None, ds=None):
    c = {k: _cut(v, cu, 1) if k in ("x", "r", "i", "z") else v for k, v in x.items()}
    return R.recur(c["x"], c["r"], c["i"], c["decay"], c["r_bias"], c["i_bias"], c["z"], c["initial_state"], cu, rate, _cut(dout, cu, 1), ds)


RECUR = [  # dtype, D, sequences, options
    (BF, 64, (1, 40), {}), (FF, 70, (2, 19), {}), (HF, 128, (2, 33), {}), (BF, 8, (1, 1), {}), (FF, 3, (3, 2), {}), (BF, 1, (1, 5), {}),
    # around the tiles of a wave, the rounds of a block, the chunks of a call
    (BF, 66, (1, 15), {}), (BF, 66, (1, 16), {}), (HF, 30, (2, 17), {}), (FF, 10, (1, 8), {}), (FF, 10, (2, 9), {}), (BF, 130, (1, 64), {}),
    (BF, 130, (1, 65), {}), (HF, 20, (1, 127), {}), (HF, 20, (1, 128), {}), (HF, 20, (1, 129), {}), (FF, 20, (3, 63), {}), (FF, 21, (2, 130), {}),
    (BF, 40, (1, 513), {}), (BF, 16, (2, 1100), {}), (FF, 2, (1, 2500), {}),
    (BF, 80, (2, 130), dict(gate=False)), (HF, 36, (2, 70), dict(bias=False)), (BF, 65, (1, 100), dict(strided=True)), (FF, 64, (1, 90), dict(init=False)),
    (HF, 33, (2, 16), dict(strided=True, gate=False)), (BF, 260, (40, 20), {}), (FF, 5, ("packed", [0, 0, 3], 0), {}),
    (FF, 72, ("packed", [0, 1, 5, 0, 170, 33, 2], 9), {}), (BF, 130, ("packed", [300, 0, 1, 129], 50), {}), (HF, 12, ("packed", [1], 0), dict(bias=False)),
    (FF, 36, PACKED, dict(gate=False, init=False)), (BF, 68, PACKED, dict(strided=True)), (HF, 64, ("packed", [2] * 65, 3), {}),
    (BF, 20, ("packed", [0, 0], 70), {}), (FF, 16, ("packed", [1] * 30 + [1500] + [0] * 5, 2), {}), (BF, 32, ("packed", [64, 128, 256, 63, 1], 200), {}),
    # few long sequences, and many of some tokens: the chunks of a gradient differ
    (BF, 34, ("packed", [600, 1, 0, 500], 3), {}), (FF, 9, ("packed", [1030], 0), dict(gate=False)), (HF, 17, ("packed", [16, 17, 15, 31, 33] * 14, 1), {}),
    # decays so small that nearly nothing is forgotten or enters, and so large that nothing is kept
    (FF, 32, (1, 200), dict(slow=16.0)), (BF, 32, (1, 200), dict(slow=-40.0)), (FF, 32, (2, 200), dict(slow=100.0)),
]


@pytest.mark.parametrize("dtype,D,seqs,opt", RECUR)
def test_recur(dtype, D, seqs, opt):
    log(f"[recur] {dtype} D={D} {seqs} {opt}")
    g = _gen(D * 100 + seqs[0] if seqs[0] != "packed" else D)
    lead, cu, n = _lead(seqs)
    x = _recur_inputs(g, lead, n, D, dtype, **opt)
    dout = _rows(g, lead, D, dtype, opt.get("strided", False))
    ds = torch.randn(n, D, generator=g).cuda()
    cud, rate = None if cu is None else cu.cuda(), 8.0 if D % 3 else 2.5
    o = m.mamba_recur_fwd(**x, cu_seqlens=cud, rate=rate, return_state=True)
    gr = m.mamba_recur_bwd(dout, **x, dstate=ds, cu_seqlens=cud, rate=rate)
    torch.cuda.synchronize()
    ref, bound = _reference(x, cu, rate, dout, ds)
    got = {k: _cut(v, cu, 1) if k in ("dx", "dr", "di", "dz") else v for k, v in gr._asdict().items()}
    for k, src in (("dr_bias", "r_bias"), ("di_bias", "i_bias"), ("dz", "z"), ("dinitial_state", "initial_state")):
        assert (got[k] is None) == (x[src] is None), k
    got.update(out=_cut(o.out, cu, 1), state=o.state)
    log(f"  worst {R.check(got, ref, bound, (dtype, D, seqs)):.3f}")
    for t in (o.out, gr.dx, gr.dr, gr.di, gr.dz):
        _tail_is(t, cu, 0.0)
    # a caller's output: written in place, rows behind the last sequence left as they were
    out = torch.full((*lead, D), 7.0, dtype=dtype, device="cuda")
    again = m.mamba_recur_fwd(**x, cu_seqlens=cud, rate=rate, out=out)
    assert again.out is out and again.state is None
    assert _same(_cut(out, cu, 1), _cut(o.out, cu, 1))
    _tail_is(out, cu, 7.0)
    # equal inputs give equal bits, whatever lies in the workspace
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    for k, t in zip(gr._fields, m.mamba_recur_bwd(dout, **x, dstate=ds, cu_seqlens=cud, rate=rate, workspace=ws)):
        assert _same(t, getattr(gr, k)), k


@pytest.mark.parametrize("idx", STEP_IDX)
@pytest.mark.parametrize("dtype,D,pad,gate", [(BF, 72, 0, True), (FF, 21, 3, True), (HF, 600, 2, False)])
def test_recur_step(dtype, D, pad, gate, idx):
    g = _gen(D)
    n, slots = 3 if idx is None else len(idx), 70
    pool = torch.randn(slots, D + pad, generator=g).cuda()
    state, before = pool[:, :D], pool.clone()
    x = _recur_inputs(g, (n,), 1, D, dtype, gate=gate, init=False, strided=bool(pad))
    x.pop("initial_state")
    ind = None if idx is None else torch.tensor(idx, dtype=torch.int32).cuda()
    out = m.mamba_recur_step(state=state, state_indices=ind, **x)
    torch.cuda.synchronize()
    want, bound, after = torch.zeros(n, D, dtype=torch.float64), torch.zeros(n, D, dtype=torch.float64), before.cpu().double()
    err = torch.zeros_like(after)
    par = (x["decay"], x["r_bias"], x["i_bias"])
    for row, k in _serial(idx, n, slots):
        one = [x[name][row:row + 1, None] for name in ("x", "r", "i")]
        ref, b = R.recur(*one, *par, None if x["z"] is None else x["z"][row:row + 1, None], after[k:k + 1, :D].clone(), None, 8.0)
        want[row] = ref["out"][0, 0]
        # the state's bound is carried over to the next token of the slot; a gate multiplies it by less than |z|
        bound[row] = b["out"][0, 0] + err[k, :D] * (1 if x["z"] is None else x["z"][row].double().abs().cpu())
        after[k, :D] = ref["state"][0]
        err[k, :D] += b["state"][0]
    R.check({"out": out}, {"out": want}, {"out": bound}, idx)
    R.check({"pool": pool}, {"pool": after}, {"pool": err}, idx)
    skipped = [] if idx is None else [k for k, v in enumerate(idx) if not 0 <= v < slots]
    assert torch.equal(out[skipped], torch.zeros_like(out[skipped]))


def test_recur_step_continues_a_prompt():
    """A prompt's state goes on token by token as the longer prompt."""
    g = _gen(5)
    n, S, D = 3, 200, 96
    x = _recur_inputs(g, (n, S), n, D, FF)
    whole = m.mamba_recur_fwd(**x, return_state=True)
    cut = {k: v[:, :190] if k in ("x", "r", "i", "z") else v for k, v in x.items()}
    first = m.mamba_recur_fwd(**cut, return_state=True)
    assert torch.allclose(first.out, whole.out[:, :190], rtol=1e-4, atol=1e-6)
    state = first.state
    par = {k: x[k] for k in ("decay", "r_bias", "i_bias")}
    for t in range(190, S):
        out = m.mamba_recur_step(x["x"][:, t], x["r"][:, t], x["i"][:, t], state, z=x["z"][:, t], **par)
        assert torch.allclose(out, whole.out[:, t], rtol=1e-4, atol=1e-6)
    assert torch.allclose(state, whole.state, rtol=1e-4, atol=1e-6)


def test_recur_special_values():
    """NaN and infinities reach their own channel's later tokens and no other channel, sequence or earlier token."""
    g = _gen(9)
    x = _recur_inputs(g, (2, 300), 2, 40, FF)
    clean = m.mamba_recur_fwd(**x, return_state=True)
    for name, value in (("x", float("nan")), ("x", float("inf")), ("r", float("nan")), ("i", float("nan")), ("z", float("nan"))):
        y = {k: v if v is None else v.clone() for k, v in x.items()}
        y[name][1, 130, 7] = value
        got = m.mamba_recur_fwd(**y, return_state=True)
        mask = torch.zeros(2, 300, 40, dtype=torch.bool, device="cuda")
        mask[1, 130:, 7] = True
        if name == "z":
            mask[1, 131:, 7] = False
        assert torch.equal(got.out[~mask], clean.out[~mask]), name
        assert not torch.isfinite(got.out[mask]).any(), (name, value)
    # open and closed gates: exp(l) between 2^-rate and 1
    y = {k: v if v is None else v.clone() for k, v in x.items()}
    y["r"][:, :, 0], y["r"][:, :, 1] = float("-inf"), float("inf")
    y["i"][:, :, 2] = float("-inf")
    got = m.mamba_recur_fwd(**y, return_state=True)
    assert torch.equal(got.state[:, 0], x["initial_state"][:, 0])       # nothing is forgotten, nothing enters
    assert torch.isfinite(got.out).all()
    gr = m.mamba_recur_bwd(torch.randn(2, 300, 40, generator=g).cuda(), **y)
    assert all(torch.isfinite(t).all() for t in gr if t is not None)


# ---------------------------------------------------------------- residual addition and norm
def _norm_inputs(g, rows, D, dtype, stream, add, strided):
    x = _rows(g, rows, D, dtype, strided)
    res = _rows(g, rows, D, stream, strided, 3.0) if add else None
    return x, res, (1 + 0.2 * torch.randn(D, generator=g)).cuda()


NORM = [  # dtype, stream, leading axes, D, residual, dropout, strided
    (BF, BF, (7,), 64, True, 0.0, False), (BF, FF, (5,), 128, True, 0.0, False), (HF, HF, (3,), 136, True, 0.0, False), (FF, FF, (9,), 512, True, 0.0, False),
    (BF, BF, (1,), 1, True, 0.0, False), (HF, FF, (2,), 7, True, 0.0, True), (BF, BF, (2, 3), 520, True, 0.0, True), (FF, FF, (5,), 1003, True, 0.0, False),
    (BF, BF, (3,), 1024, False, 0.0, False), (BF, FF, (3,), 1032, False, 0.0, False), (HF, HF, (33,), 2048, True, 0.0, False), (BF, FF, (2,), 4096, True, 0.0, False),
    (HF, HF, (2,), 4104, True, 0.0, False), (FF, FF, (2,), 8192, True, 0.0, False), (BF, BF, (2,), 8200, True, 0.0, False), (FF, FF, (1,), 16384, True, 0.0, False),
    (BF, FF, (2,), 16381, True, 0.0, True), (BF, BF, (19,), 40, True, 0.3, False), (BF, FF, (6,), 72, True, 0.1, False), (HF, HF, (4,), 65, False, 0.5, True),
    (FF, FF, (3,), 260, True, 0.9, False), (BF, BF, (2,), 520, False, 0.1, False), (FF, FF, (700,), 24, True, 0.0, False), (BF, BF, (5000,), 16, True, 0.0, False),
    (HF, FF, (300,), 200, True, 0.25, False),
    # blocks of 3, 5, 9 and 16 waves that take several rows each, and rows of two accesses a thread
    (BF, BF, (1700,), 1100, True, 0.0, False), (HF, FF, (1300,), 2056, True, 0.1, False), (BF, BF, (600,), 4104, True, 0.2, False),
    (FF, FF, (520,), 8190, True, 0.0, True), (BF, FF, (530,), 8200, True, 0.1, False), (FF, FF, (600,), 8201, True, 0.0, False),
]
SEED = (0x1234567_89ABCDEF, -0x0FEDCBA9_87654321)


def _mask(rows, D, drop):
    if not drop:
        return None, 1.0
    cut = int(drop * 65536 + 0.5)
    return R.kept(SEED, rows, D, cut), 65536 / (65536 - cut)


@pytest.mark.parametrize("dtype,stream,lead,D,add,drop,strided", NORM)
def test_add_norm(dtype, stream, lead, D, add, drop, strided):
    log(f"[add_norm] {dtype} {stream} {lead} D={D} add={add} drop={drop} strided={strided}")
    g = _gen(D + lead[0])
    x, res, w = _norm_inputs(g, lead, D, dtype, stream, add, strided)
    rows = x.numel() // D
    mask, f = _mask(rows, D, drop)
    seed = torch.tensor(SEED).cuda() if drop else None
    args = dict(eps=1e-5, dropout=drop, seed=seed)
    o = m.mamba_add_norm_fwd(x, w, res, sum_dtype=stream, **args)
    torch.cuda.synchronize()
    ref, bound = R.add_norm(x, w, res, 1e-5, mask, f)
    assert o.sum.dtype == stream and o.out.dtype == dtype and o.scale is None
    log(f"  worst {R.check(dict(sum=o.sum, out=o.out), ref, bound, 'forward'):.3f}")
    if not add and not drop and stream == dtype:
        assert o.sum is x
    out = torch.empty_like(o.out)
    assert m.mamba_add_norm_fwd(x, w, res, sum_dtype=stream, out=out, **args).out is out and _same(out, o.out)
    # gradients, from the stored sum
    dout, ds = _rows(g, lead, D, dtype, strided), _rows(g, lead, D, stream, strided)
    for late in (ds, None):
        gr = m.mamba_add_norm_bwd(dout, o.sum, w, late, residual=add, **args)
        torch.cuda.synchronize()
        gref, gbound = R.add_norm_grads(dout, o.sum, w, late, 1e-5, mask, f)
        assert (gr.dresidual is None) == (not add)
        if add:
            assert gr.dresidual.dtype == stream and (gr.dresidual is gr.dx) == (not drop and stream == dtype)
        assert gr.dx.dtype == dtype
        log(f"  worst {R.check(gr._asdict(), gref, gbound, 'backward'):.3f}")
    again = m.mamba_add_norm_bwd(dout, o.sum, w, None, residual=add, workspace=torch.full((1 << 25,), 255, dtype=torch.uint8, device="cuda"), **args)
    for a, b in zip(again, gr):
        assert _same(a, b)


@pytest.mark.parametrize("dtype,D,lead", [(BF, 64, (3,)), (HF, 1003, (5,)), (FF, 300, (4,)), (BF, 2048, (9,)), (FF, 33, (2, 2)), (BF, 8200, (2,)), (HF, 16384, (1,)),
                                          (BF, 1, (3,)), (BF, 640, (17,)), (HF, 100, (50,)), (BF, 1100, (6,)), (FF, 2056, (3,)), (BF, 8192, (2,)), (HF, 256, (11,))])
@pytest.mark.parametrize("kind", [E4, I8])
def test_add_norm_in_8_bits(dtype, D, lead, kind):
    g = _gen(D)
    x, res, w = _norm_inputs(g, lead, D, dtype, FF, True, False)
    x[..., D // 2:] *= 30           # blocks of different size
    ref, bound = R.add_norm(x, w, res, 1e-5)
    y, e = ref["out"].reshape(-1, D), bound["out"].reshape(-1, D)
    rows = y.shape[0]
    for block in (None, 32, 64, 128, 256):
        o = m.mamba_add_norm_fwd(x, w, res, out_dtype=kind, block=block)
        torch.cuda.synchronize()
        assert o.out.dtype == kind and o.out.shape == x.shape and o.scale.shape == (*lead, -(-D // block) if block else 1)
        top = 448.0 if kind == E4 else 127.0
        s, cs, wide, cw = R.scales(ref["out"], bound["out"], block, top)
        R.check({"scale": o.scale.reshape(rows, -1)}, {"scale": s}, {"scale": s * cs}, (kind, block))
        t = y / wide
        near = R.U * (t.abs() * (cw + 3) + e / wide)
        half = torch.maximum(t.abs() * 2.0 ** -4, torch.full_like(t, 2.0 ** -10)) if kind == E4 else torch.full_like(t, 0.5)
        q = o.out.reshape(-1, D).cpu().double()
        assert ((q - t).abs() <= half + near).all(), (kind, block, float(((q - t).abs() - half - near).max()))
        assert float(q.abs().max()) <= top


def test_add_norm_special_rows():
    """Rows of zeros, of one NaN, of one infinity, in each output; dropped elements do not count, whatever they hold."""
    D = 512
    x, w = torch.randn(5, D, generator=_gen(1)).cuda(), torch.ones(D).cuda()
    x[0] = 0
    x[1, 100], x[2, 300] = float("nan"), float("inf")
    o = m.mamba_add_norm_fwd(x, w)
    assert torch.equal(o.out[0], x[0]) and torch.isnan(o.out[1]).all() and torch.isnan(o.out[2, 300]) and float(o.out[2, :300].abs().max()) == 0
    for kind in (E4, I8):
        for block in (None, 128):
            q = m.mamba_add_norm_fwd(x, w, out_dtype=kind, block=block)
            assert float(q.out[0].float().abs().max()) == 0 and torch.isfinite(q.scale[0]).all()
            assert torch.isnan(q.scale[1]).all() and torch.isnan(q.scale[2]).tolist() == ([True] if block is None else [False, False, True, False])
            assert torch.isnan(q.out[1].float()).all() if kind == E4 else float(q.out[1].float().abs().max()) == 0
            assert torch.isfinite(q.scale[3:]).all()
    seed = torch.tensor(SEED).cuda()
    keep = R.kept(SEED, 5, D, 32768).cuda()
    bad = torch.where(keep, torch.randn(5, D, generator=_gen(2)).cuda(), torch.full((5, D), float("nan")).cuda())
    o = m.mamba_add_norm_fwd(bad, w, dropout=0.5, seed=seed)
    assert torch.isfinite(o.out).all() and torch.equal(o.sum == 0, ~keep)


def test_dropout_by_seed():
    """Another seed or offset drops others; the same drops the same, in either direction, whatever the strides and the batch's shape."""
    D, rows = 264, 40
    one, w = torch.ones(rows, D, device="cuda"), torch.ones(D, device="cuda")

    def kept(x, *seed):
        return m.mamba_add_norm_fwd(x, w, dropout=0.3, seed=torch.tensor(seed).cuda()).sum != 0
    base = kept(one, 5, 6)
    assert torch.equal(base.cpu(), R.kept((5, 6), rows, D, 19661))
    assert torch.equal(base, kept(one.view(4, 10, D), 5, 6).view(rows, D)) and torch.equal(base, kept(torch.ones(rows, D + 3, device="cuda")[:, 1:D + 1], 5, 6))
    for other in ((6, 6), (5, 7), (5 + (1 << 40), 6), (5, 6 + (1 << 40))):
        assert 0.3 < float((kept(one, *other) != base).float().mean()) < 0.55
    v = torch.randn(rows, D, generator=_gen(0)).cuda()
    g = m.mamba_add_norm_bwd(torch.zeros_like(v), v, w, torch.ones_like(v), dropout=0.3, seed=torch.tensor((5, 6)).cuda())
    assert torch.equal(g.dx != 0, base) and torch.equal(g.dresidual, torch.ones_like(v))


# ---------------------------------------------------------------- streams, graphs, a run together
def test_on_another_stream():
    g = _gen(3)
    x = _recur_inputs(g, (2, 400), 2, 130, BF)
    n = torch.randn(50, 700, generator=g).to(BF).cuda()
    w = torch.ones(700).cuda()
    torch.cuda.synchronize()
    here = (m.mamba_recur_fwd(**x, return_state=True), m.mamba_add_norm_fwd(n, w, n, out_dtype=E4, block=32))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        there = (m.mamba_recur_fwd(**x, return_state=True), m.mamba_add_norm_fwd(n, w, n, out_dtype=E4, block=32))
    s.synchronize()
    torch.cuda.synchronize()
    assert _same(here[0].out, there[0].out) and _same(here[0].state, there[0].state)
    assert torch.equal(here[1].out.view(I8), there[1].out.view(I8)) and _same(here[1].scale, there[1].scale)


def _training_step(x, w, par, seed, dout):
    """Addition with dropout, norm, recurrence, and back: a block's operators without its products."""
    a = m.mamba_add_norm_fwd(x["x"], w, x["res"], dropout=0.2, seed=seed)
    o = m.mamba_recur_fwd(a.out, x["r"], x["i"], **par, z=x["z"], return_state=True)
    g = m.mamba_recur_bwd(dout, a.out, x["r"], x["i"], **par, z=x["z"])
    b = m.mamba_add_norm_bwd(g.dx, a.sum, w, dout.to(a.sum.dtype), dropout=0.2, seed=seed)
    return [t for t in (*a, *o, *g, *b) if t is not None]


def test_captured_training_step():
    """Forward and backward of both operators in one graph; replays take the seed and inputs that lie there then, and agree with
    eager calls, with eager work in between."""
    g = _gen(11)
    B, S, D = 2, 300, 264
    new = lambda t: torch.randn(B, S, D, generator=g).to(t).cuda()  # noqa: E731
    x = dict(x=new(BF), r=new(BF), i=new(BF), z=new(BF), res=new(FF))
    par = dict(decay=(torch.randn(D, generator=g) - 3).cuda(), r_bias=torch.randn(D, generator=g).cuda(), i_bias=torch.randn(D, generator=g).cuda())
    w, seed, dout = torch.rand(D, generator=g).cuda() + 0.5, torch.tensor([1, 2]).cuda(), new(BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _training_step(x, w, par, seed, dout)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _training_step(x, w, par, seed, dout)
    sums = []
    for k in range(4):
        seed.copy_(torch.tensor([k, 100 * k]))
        x["x"].copy_(new(BF))
        graph.replay()
        torch.cuda.synchronize()
        eager = _training_step(x, w, par, seed, dout)
        assert all(_same(a, b) for a, b in zip(held, eager)), k
        sums.append((held[1] == x["res"]).sum().item())
    assert len(set(sums)) > 1


def test_two_graphs_with_one_workspace_of_their_own_each():
    """Two captured calls replayed on two streams at once, each with its own workspace."""
    g = _gen(12)
    xs = [_recur_inputs(g, (2, 500), 2, 128, BF) for _ in range(2)]
    douts = [torch.randn(2, 500, 128, generator=g).to(BF).cuda() for _ in range(2)]
    want = [m.mamba_recur_bwd(d, **x) for d, x in zip(douts, xs)]
    graphs, held = [], []
    for d, x in zip(douts, xs):
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        q = torch.cuda.CUDAGraph()
        with torch.cuda.graph(q):
            held.append((m.mamba_recur_bwd(d, **x, workspace=ws), ws))
        graphs.append(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for q, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                q.replay()
        torch.cuda.synchronize()
        for (got, _), ref in zip(held, want):
            assert all(_same(a, b) for a, b in zip(got, ref))


class _Stack:
    """Two recurrent blocks around a residual stream, in float64-free torch for the products: norm of the stream -> projections ->
    short convolution -> recurrence -> projection -> addition and the next norm."""

    def __init__(self, g, D, E, dtype):
        t = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale)  # noqa: E731
        self.dtype = dtype
        self.blocks = [dict(norm=(1 + 0.1 * t(D)).cuda(), wx=(t(D, 4 * E) / D ** 0.5).to(dtype).cuda(), conv=(t(E, 4) / 2).cuda(), decay=(t(E) - 4).cuda(),
                            rb=t(E).cuda(), ib=t(E).cuda(), out=(t(E, D) / E ** 0.5).to(dtype).cuda()) for _ in range(2)]
        self.last = (1 + 0.1 * t(D)).cuda()
        self.E = E

    def prompt(self, x):
        """x [B, S, D]: (last norm's output, states of each block)."""
        total, add, states = None, x, []
        for b in self.blocks:
            o = m.mamba_add_norm_fwd(add, b["norm"], total, sum_dtype=torch.float32)
            total = o.sum
            u, r, i, z = (o.out @ b["wx"]).split(self.E, -1)
            c = m.mamba_conv_fwd(u, b["conv"], activation="silu", return_state=True)
            h = m.mamba_recur_fwd(c.out, r, i, b["decay"], b["rb"], b["ib"], z, return_state=True)
            states.append([c.state, h.state])
            add = h.out @ b["out"]
        return m.mamba_add_norm_fwd(add, self.last, total).out, states

    def token(self, x, states):
        total, add = None, x
        for b, s in zip(self.blocks, states):
            o = m.mamba_add_norm_fwd(add, b["norm"], total, sum_dtype=torch.float32)
            total = o.sum
            u, r, i, z = (o.out @ b["wx"]).split(self.E, -1)
            c = m.mamba_conv_step(u, s[0], b["conv"], activation="silu")
            h = m.mamba_recur_step(c, r, i, s[1], b["decay"], b["rb"], b["ib"], z)
            add = h @ b["out"]
        return m.mamba_add_norm_fwd(add, self.last, total).out


def test_stack_of_blocks():
    """A prompt, then tokens one by one, as the longer prompt gives them, in float32 (rounding of the products alone differs)."""
    g = _gen(21)
    stack = _Stack(g, 48, 80, FF)
    x = torch.randn(2, 150, 48, generator=g).cuda()
    whole, _ = stack.prompt(x)
    got, states = stack.prompt(x[:, :140].contiguous())
    # 1e-3: some thirty products and sums of 48 to 320 terms in a row, each within 320 * 2^-24 = 2e-5 of its terms' size
    assert torch.allclose(got, whole[:, :140], rtol=1e-3, atol=1e-3)
    for t in range(140, 150):
        assert torch.allclose(stack.token(x[:, t].contiguous(), states), whole[:, t], rtol=1e-3, atol=1e-3)


def test_stack_gradient():
    """The operators' backward calls chained by hand through one block and its addition: against 64-bit automatic
    differentiation of the same formulas."""
    g = _gen(22)
    B, S, D = 2, 70, 24
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res, r, i, z, dout = (t(B, S, D) for _ in range(6))
    w1, w2, decay, rb, ib = 1 + 0.1 * t(D), 1 + 0.1 * t(D), t(D) - 3, t(D), t(D)
    dev = lambda *a: [v.cuda() for v in a]  # noqa: E731
    cx, cres, cr, ci, cz, cd, c1, c2, cdec, crb, cib = dev(x, res, r, i, z, dout, w1, w2, decay, rb, ib)
    a = m.mamba_add_norm_fwd(cx, c1, cres)
    h = m.mamba_recur_fwd(a.out, cr, ci, cdec, crb, cib, cz)
    b = m.mamba_add_norm_fwd(h.out, c2, a.sum)
    gb = m.mamba_add_norm_bwd(cd, b.sum, c2)
    gh = m.mamba_recur_bwd(gb.dx, a.out, cr, ci, cdec, crb, cib, cz)
    ga = m.mamba_add_norm_bwd(gh.dx, a.sum, c1, gb.dresidual)
    leaves = [v.double().requires_grad_() for v in (x, res, r, i, z, w1, w2, decay, rb, ib)]
    lx, lres, lr, li, lz, l1, l2, ldec, lrb, lib = leaves
    v = lx + lres
    n1 = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * l1
    hh, ys = torch.zeros(B, D, dtype=torch.float64), []
    for k in range(S):
        ak = torch.exp(-8 * torch.nn.functional.softplus(ldec) * torch.sigmoid(lr[:, k] + lrb))
        hh = ak * hh + torch.sqrt(1 - ak * ak) * torch.sigmoid(li[:, k] + lib) * n1[:, k]
        ys.append(hh * torch.nn.functional.silu(lz[:, k]))
    v2 = torch.stack(ys, 1) + v
    out = v2 / torch.sqrt((v2 * v2).mean(-1, keepdim=True) + 1e-5) * l2
    want = torch.autograd.grad((out * dout.double()).sum(), leaves)
    got = [ga.dx, ga.dresidual, gh.dr, gh.di, gh.dz, ga.dweight, gb.dweight, gh.ddecay, gh.dr_bias, gh.di_bias]
    for k, (p, q) in enumerate(zip(got, want)):
        # 2^-24 times some thousand roundings (70 tokens, two norms, sums over 140 tokens) of terms of the gradient's size
        assert float((p.cpu().double() - q).norm() / q.norm()) < 4000 * R.U, k


def test_recur_with_far_tokens():
    """Tokens 2^26 elements and more apart (a time-major buffer of a huge batch) are copied, those just below are read in place."""
    g = _gen(41)
    D, far = 24, (1 << 26) + 8
    x = _recur_inputs(g, (1, 3), 1, D, BF)
    want = m.mamba_recur_fwd(**x, return_state=True)
    dout = torch.randn(1, 3, D, generator=g).to(BF).cuda()
    grads = m.mamba_recur_bwd(dout, **x)
    room = torch.empty(2 * far + D, dtype=BF, device="cuda")
    for stride in (far, 1 << 26, (1 << 26) - 8):
        y = room.as_strided((1, 3, D), (0, stride, 1))
        y.copy_(x["r"])
        got = m.mamba_recur_fwd(**{**x, "r": y}, return_state=True)
        assert _same(got.out, want.out) and _same(got.state, want.state)
        assert all(_same(a, b) for a, b in zip(m.mamba_recur_bwd(dout, **{**x, "r": y}), grads))


def test_recur_with_repeated_tokens():
    """One row for every token (stride 0), and rows that overlap."""
    g = _gen(42)
    D, S = 40, 150
    x = _recur_inputs(g, (2, S), 2, D, HF)
    one = torch.randn(2, 1, D, generator=g).to(HF).cuda()
    line = torch.randn(S + D, generator=g).to(HF).cuda()
    dout = torch.randn(2, S, D, generator=g).to(HF).cuda()
    for y in (one.expand(2, S, D), line.as_strided((2, S, D), (0, 1, 1))):
        a, b = ({**x, "x": v, "z": v} for v in (y, y.contiguous()))
        assert _same(m.mamba_recur_fwd(**a).out, m.mamba_recur_fwd(**b).out)
        assert all(_same(p, q) for p, q in zip(m.mamba_recur_bwd(dout, **a), m.mamba_recur_bwd(dout, **b)))


@pytest.mark.parametrize("rate,decay", [(3e38, [0.0, 3.0, 50.0, 3e38, -20.0]), (8.0, [1e31, 3e38, 5e37, 1e36, 2e30])])
def test_recur_of_decays_without_measure(rate, decay):
    """rate softplus(decay) up to fp32's range and beyond it: nothing is kept, nothing but the token itself has a gradient, and no
    product of zero and infinity comes up."""
    g = _gen(43)
    D, S = len(decay), 150
    x = _recur_inputs(g, (2, S), 2, D, FF)
    x["decay"] = torch.tensor(decay, device="cuda")
    x["initial_state"] *= 1e6
    dout, ds = _rows(g, (2, S), D, FF, False), torch.randn(2, D, generator=g).cuda()
    o, gr = m.mamba_recur_fwd(**x, rate=rate, return_state=True), m.mamba_recur_bwd(dout, **x, dstate=ds, rate=rate)
    v = {k: t.double() for k, t in x.items()}
    si, sz = torch.sigmoid(v["i"] + v["i_bias"]), torch.sigmoid(v["z"])
    h = si * v["x"]
    dh = dout.double() * v["z"] * sz
    dh[:, -1] += ds
    # sigmoids of arguments below 8: (8 * 1.5 + 4) u each; up to three of them and six products
    near = lambda a, b, size: bool(((a.double() - b).abs() <= 60 * R.U * size.abs()).all())  # noqa: E731
    assert near(o.out, h * v["z"] * sz, h * v["z"] * sz) and near(o.state, h[:, -1], h[:, -1])
    size = dout.double().abs() * v["z"].abs() * sz
    size[:, -1] += ds.abs()
    assert near(gr.dx, dh * si, size * si) and near(gr.di, dh * h * (1 - si), size * h)
    dz = dout.double() * h
    assert near(gr.dz, dz * (sz + v["z"] * sz * (1 - sz)), dz * (1 + v["z"].abs()))
    for t in (gr.dr, gr.ddecay, gr.dr_bias, gr.dinitial_state):
        assert not t.any()
    s = torch.zeros(2, D, device="cuda")
    one = {k: t[:, 0].contiguous() for k, t in x.items() if k in "xriz"}
    y = m.mamba_recur_step(state=s, **one, decay=x["decay"], r_bias=x["r_bias"], i_bias=x["i_bias"], rate=rate)
    assert _same(y, o.out[:, 0]) and near(s, h[:, 0], h[:, 0])


@pytest.mark.parametrize("dtype,D,S,gate", [(BF, 2048, 2048, True), (HF, 2047, 2050, False), (FF, 1030, 2000, True), (FF, 1024, 2010, False), (HF, 1984, 2050, False)])
def test_recur_gradient_larger_than_the_cache(dtype, D, S, gate):
    """A call beyond the last-level cache's size gives a sequence's gradients the bits that a call for the sequence alone gives them."""
    g = torch.Generator(device="cuda").manual_seed(51)
    n = 5
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {k: new(n, S, D).to(dtype) for k in ("x", "r", "i")}
    x["z"] = new(n, S, D).to(dtype) if gate else None
    x.update(decay=new(D) - 3, r_bias=new(D), i_bias=None, initial_state=new(n, D))
    dout, ds = new(n, S, D).to(dtype), new(n, D)
    assert n * S * D * (9 if gate else 7) * dout.element_size() > 256 << 20
    whole = m.mamba_recur_bwd(dout, **x, dstate=ds)
    total = torch.zeros(D, dtype=torch.float64, device="cuda")
    for k in range(n):
        one = m.mamba_recur_bwd(dout[k:k + 1], **{a: v if v is None or v.dim() == 1 else v[k:k + 1] for a, v in x.items()}, dstate=ds[k:k + 1])
        for name in ("dx", "dr", "di", "dz", "dinitial_state"):
            a, b = getattr(whole, name), getattr(one, name)
            assert (a is None and b is None) or _same(a[k:k + 1], b), name
        total += one.ddecay.double()
    # sums of n * S terms in fp32: their errors are those of some hundred roundings of the terms' size, sqrt(n S) of which remain
    assert float((whole.ddecay.double() - total).norm() / total.norm()) < 300 * R.U


@pytest.mark.parametrize("dtype,D,S,gate", [(BF, 1984, 3001, True), (HF, 517, 13001, False), (FF, 1001, 3001, True), (FF, 1056, 3201, False), (HF, 704, 10001, False)])
def test_recur_larger_than_the_cache(dtype, D, S, gate):
    """A call beyond the last-level cache's size gives a sequence the bits that a call for the sequence alone gives it."""
    g = torch.Generator(device="cuda").manual_seed(52)
    n = 5
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {k: new(n, S, D).to(dtype) for k in ("x", "r", "i")}
    x["z"] = new(n, S, D).to(dtype) if gate else None
    x.update(decay=new(D) - 3, r_bias=None, i_bias=new(D), initial_state=new(n, D))
    assert n * S * D * (5 if gate else 4) * x["x"].element_size() > 256 << 20
    whole = m.mamba_recur_fwd(**x, return_state=True)
    for k in range(n):
        one = m.mamba_recur_fwd(**{a: v if v is None or v.dim() == 1 else v[k:k + 1] for a, v in x.items()}, return_state=True)
        assert _same(whole.out[k:k + 1], one.out) and _same(whole.state[k:k + 1], one.state), k


@pytest.mark.parametrize("packed", [False, True])
def test_recur_beyond_32_bits(packed):
    """More than 2^31 elements in a tensor: the last sequence gets the bits that a call for it alone gets."""
    g = torch.Generator(device="cuda").manual_seed(53)
    S, D = 1 << 20, 1032
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {k: torch.empty(2, S, D, dtype=BF, device="cuda") for k in ("x", "r", "i", "z")}
    for t in x.values():
        assert t.numel() > 1 << 31
        t[0] = 0.5
        t[1].view(64, S // 64, D)[:] = new(S // 64, D)
    dout = x["z"]                   # any tensor of its size does
    par, init = dict(decay=new(D) - 3, r_bias=new(D)), new(2, D)
    cu = torch.tensor([0, S, 2 * S], dtype=torch.int32, device="cuda") if packed else None
    flat = (lambda t: t.view(-1, D)) if packed else (lambda t: t)
    whole = {k: flat(t) for k, t in x.items()}
    one = {k: t[1] if packed else t[1:] for k, t in x.items()}
    args = dict(cu_seqlens=cu), dict(cu_seqlens=None if cu is None else cu[:2].contiguous())
    a = m.mamba_recur_fwd(**whole, **par, initial_state=init, return_state=True, **args[0])
    b = m.mamba_recur_fwd(**one, **par, initial_state=init[1:], return_state=True, **args[1])
    assert _same(a.out.view(2, S, D)[1], b.out.view(S, D)) and _same(a.state[1:], b.state)
    del a, b
    a = m.mamba_recur_bwd(flat(dout), **whole, **par, initial_state=init, dstate=init, **args[0])
    b = m.mamba_recur_bwd(one["z"], **one, **par, initial_state=init[1:], dstate=init[1:], **args[1])
    for k in ("dx", "dr", "di", "dz"):
        assert _same(getattr(a, k).view(2, S, D)[1], getattr(b, k).view(S, D)), k
    assert _same(a.dinitial_state[1:], b.dinitial_state)


def test_recur_step_from_a_pool_beyond_32_bits():
    g = torch.Generator(device="cuda").manual_seed(55)
    D = 1032
    slots = (1 << 31) // D + 3
    pool = torch.empty(slots, D, device="cuda")
    pool[-1].normal_(generator=g)
    alone = pool[-1:].clone()
    x = [torch.randn(1, D, generator=g, device="cuda").to(HF) for _ in range(4)]
    decay = torch.randn(D, generator=g, device="cuda")
    y = m.mamba_recur_step(x[0], x[1], x[2], pool, decay, z=x[3], state_indices=torch.tensor([slots - 1], dtype=torch.int32).cuda())
    assert _same(y, m.mamba_recur_step(x[0], x[1], x[2], alone, decay, z=x[3])) and _same(pool[-1], alone[0])


def test_add_norm_beyond_32_bits():
    g = torch.Generator(device="cuda").manual_seed(54)
    D, rows = 1032, (1 << 21) + 300
    x, res, w = torch.zeros(rows, D, dtype=BF, device="cuda"), torch.zeros(rows, D, dtype=BF, device="cuda"), torch.rand(D, generator=g, device="cuda") + 0.5
    assert x.numel() > 1 << 31
    for t in (x, res):
        t[-300:] = torch.randn(300, D, generator=g, device="cuda")
    for kw in ({}, dict(out_dtype=E4, block=64)):
        a, b = m.mamba_add_norm_fwd(x, w, res, **kw), m.mamba_add_norm_fwd(x[-300:].clone(), w, res[-300:].clone(), **kw)
        assert _same(a.sum[-300:], b.sum) and torch.equal(a.out[-300:].view(torch.uint8), b.out.view(torch.uint8))
        assert a.scale is None or _same(a.scale[-300:], b.scale)
    p, q = m.mamba_add_norm_bwd(x, res, w, x), m.mamba_add_norm_bwd(x[-300:].clone(), res[-300:].clone(), w, x[-300:].clone())
    assert _same(p.dx[-300:], q.dx)


@pytest.mark.parametrize("D,S", [(8, 1 << 14)])
def test_long_sequence_of_few_channels(D, S):
    """Many chunks of one tile, against the sequential definition."""
    g = _gen(31)
    x = _recur_inputs(g, (1, S), 1, D, BF)
    dout, ds = torch.randn(1, S, D, generator=g).to(BF).cuda(), torch.randn(1, D, generator=g).cuda()
    o = m.mamba_recur_fwd(**x, return_state=True)
    gr = m.mamba_recur_bwd(dout, **x, dstate=ds)
    ref, bound = _reference(x, None, 8.0, dout, ds)
    R.check({**gr._asdict(), "out": o.out, "state": o.state}, ref, bound, "long")
