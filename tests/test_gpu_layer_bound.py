"""The selective scan on the GPU within the bound that tests/_layer_bound.py carries through the recurrence: the plans that
long sequences take (more than 128 chunks, chunks of 32, 64 and 128 tokens, the carry by one and by four states a
thread), sequences of every length around a unit and a chunk in one packed batch, and steps of both signs."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from . import _layer_bound as Bd
from . import _layer_ref as R
from ._parity import log
from .test_gpu_layer import _cut, _gen, _lead, _need_gpu, _rows, _same, _scan_inputs, _tail_is  # noqa: F401

pytestmark = pytest.mark.gpu
BF, HF, FF = torch.bfloat16, torch.float16, torch.float32
GRADS = ("du", "ddt", "da", "db", "dc", "dd", "dz", "ddt_bias", "dinitial_state")


def compare(dtype, D, G, N, seqs, sp=True, seed=0, bias=None, **opt):
    """Forward and backward against the bound; the largest error in parts of it."""
    g = _gen(seed + D * 100 + N)
    lead, cu, n = _lead(seqs)
    x = _scan_inputs(g, lead, n, D, G, N, dtype, sp=sp, **opt)
    if bias is not None:
        x["dt_bias"] = bias * torch.randn(D, generator=g).cuda()
    dout, ds = _rows(g, lead, D, dtype, False), torch.randn(n, D, N, generator=g).cuda()
    cud = None if cu is None else cu.cuda()
    o = m.mamba_scan_fwd(**x, cu_seqlens=cud, dt_softplus=sp, return_state=True)
    gr = m.mamba_scan_bwd(dout, **x, dstate=ds, cu_seqlens=cud, dt_softplus=sp)
    torch.cuda.synchronize()
    cut = {k: _cut(v, cu, 1) if k in ("u", "dt", "b", "c", "z") else v for k, v in x.items()}
    cut["initial"] = cut.pop("initial_state")
    ref, bound = Bd.scan(**cut, cu=cu, sp=sp, dout=_cut(dout, cu, 1), dstate=ds, chunk=128)
    got = {"out": _cut(o.out, cu, 1), "state": o.state,
           **{k: _cut(v, cu, 1) if k in ("du", "ddt", "db", "dc", "dz") else v for k, v in gr._asdict().items()}}
    names = [k for k in ("out", "state") + GRADS if got[k] is not None]
    if dtype is FF and "ddt_bias" in names:
        Bd.check_sum(got["ddt_bias"], got["ddt"], n, 128)
    worst, blunt = Bd.check(got, ref, bound, [k for k in names if k not in Bd.SUMS], seqs)
    sums = Bd.check(got, ref, bound, [k for k in names if k in Bd.SUMS], seqs)
    log(f"[scan bound] {dtype} D={D} G={G} N={N} {str(seqs)[:60]} worst {worst:.3f} (median bound {blunt:.1e}), sums {sums[0]:.3f} ({sums[1]:.1e})")
    for t in (o.out, gr.du, gr.ddt, gr.db, gr.dc, gr.dz):
        _tail_is(t, cu, 0.0)
    return blunt


AROUND = ("packed", [0, 1, 15, 16, 17, 0, 31, 32, 33, 48, 64, 100, 112, 113, 127, 128, 129, 145, 256, 300, 400], 9)
CASES = [  # dtype, D, G, N, sequences
    # more than 128 chunks of a sequence, forward and backward: several rounds of the carry's waves
    (FF, 8, 1, 4, (1, 6000)), (BF, 12, 2, 16, ("packed", [4500, 3, 1100], 5)),
    # the carry by four states a thread, in a forward pass that is cut
    (FF, 512, 1, 16, (8, 150)),
    # backward in chunks of 128, 64 and 32 tokens
    (FF, 64, 64, 4, (2, 1100)), (BF, 64, 64, 16, (1, 2100)), (FF, 48, 48, 24, (1, 1500)), (HF, 40, 40, 64, (1, 1200)), (FF, 64, 64, 100, (1, 2050)),
    # lengths around a unit and a chunk, with chunks of 128, 64 and 16 tokens
    (FF, 64, 64, 8, AROUND), (BF, 32, 32, 40, AROUND), (FF, 20, 2, 16, AROUND), (HF, 64, 64, 3, AROUND),
]


@pytest.mark.parametrize("dtype,D,G,N,seqs", CASES)
def test_within_the_bound(dtype, D, G, N, seqs):
    assert compare(dtype, D, G, N, seqs) < 2e-3     # what is compared is pinned to a part in 500 of its value


@pytest.mark.parametrize("dtype,D,G,N,seqs", [(FF, 24, 3, 5, (1, 40)), (FF, 16, 1, 16, (2, 100))])
def test_steps_of_both_signs(dtype, D, G, N, seqs):
    """Without softplus, steps between -0.15 and 0.5: states shrink and grow, and stay in fp32's range."""
    assert compare(dtype, D, G, N, seqs, sp=False, bias=0.03) < 2e-2


def test_more_than_2_32_partial_sums():
    """256 times the same sequence, whose gradients of b and c have 2^32 elements: every one as the first's, and that
    within the bound. The inputs of all sequences lie in one place (a batch stride of zero)."""
    n, S, D, N = 256, 1024, 64, 128
    g = _gen(77)
    x = _scan_inputs(g, (1, S), 1, D, D, N, BF)
    dout, ds = _rows(g, (1, S), D, BF, False), torch.randn(1, D, N, generator=g).cuda()
    wide = {k: v if k in ("a", "d", "dt_bias") else v.expand(n, *v.shape[1:]) for k, v in x.items()}
    gr = m.mamba_scan_bwd(dout.expand(n, S, D), **wide, dstate=ds.expand(n, D, N), dt_softplus=True)
    for k in ("db", "dc", "du", "ddt", "dz", "dinitial_state"):
        t = getattr(gr, k)
        for i in range(1, n):
            assert torch.equal(t[i], t[0]), (k, i)
    x["initial"] = x.pop("initial_state")
    ref, bound = Bd.scan(**x, cu=None, sp=True, dout=dout, dstate=ds, chunk=128)
    got = {k: getattr(gr, k)[:1] for k in ("db", "dc", "du", "ddt", "dz", "dinitial_state")}
    log(f"[scan bound] 2^32 sums: worst {Bd.check(got, ref, bound, tuple(got))[0]:.3f}")


def _kind(x):
    """0 finite, 1 infinite, -1 minus infinite, 2 not a number."""
    x = x.detach().cpu().double()
    return torch.where(x.isnan(), 2, torch.where(x.isinf(), x.sign(), torch.zeros_like(x)).long())


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 12, 13, 16, 24, 31, 40, 100])
@pytest.mark.parametrize("dtype,D,S,what", [(FF, 5, 96, "u"), (BF, 70, 48, "dt"), (FF, 20, 32, "dout"), (BF, 6, 200, "u")])
def test_infinite_inputs(dtype, D, S, what, N):
    """One infinite input among positive ones: where the formulas give an infinity, so do the outputs and gradients, for
    any number of states; the other channels stay finite."""
    g = _gen(N)
    pos = lambda *s: (torch.rand(*s, generator=g) + 0.5)  # noqa: E731
    x = {k: pos(1, S, D).to(dtype).cuda() for k in ("u", "dt", "z")}
    x["dt"] = x["dt"] * -2                          # through the softplus: 0.05 to 0.3
    x.update({k: pos(1, S, 1, N).to(dtype).cuda() for k in ("b", "c")})
    x.update(a=-pos(D, N).cuda() * 0.2, d=pos(D).cuda(), dt_bias=torch.zeros(D).cuda(), initial_state=pos(1, D, N).cuda())
    dout, ds = pos(1, S, D).to(dtype).cuda(), pos(1, D, N).cuda()
    (dout if what == "dout" else x[what])[0, S // 3, 2] = float("inf")
    o = m.mamba_scan_fwd(**x, dt_softplus=True, return_state=True)
    gr = m.mamba_scan_bwd(dout, **x, dstate=ds, dt_softplus=True)
    got = {"out": o.out, "state": o.state, **{k: v for k, v in gr._asdict().items() if v is not None}}
    names = {**x, "initial": x["initial_state"]}
    names.pop("initial_state")
    ref = R.scan(**names, cu=None, sp=True, dout=dout, dstate=ds)
    for k, v in got.items():
        if k == "da" and S % 16 and what != "dout":    # the header allows NaN there: the tokens behind the last one count with inf * 0
            continue
        assert torch.equal(_kind(v), _kind(ref[k])), k
    assert bool((_kind(ref["du"] if what == "dout" else ref["out"]) != 0).any())
    if what == "dout":
        return
    t = S // 3
    row = {k: (v[:, t] if k in ("u", "dt", "b", "c", "z") else v) for k, v in x.items()}
    state = row.pop("initial_state").clone()
    y = m.mamba_scan_step(**row, state=state, dt_softplus=True)
    one = {k: (v[:, t:t + 1] if k in ("u", "dt", "b", "c", "z") else v) for k, v in names.items()}
    ref = R.scan(**one, cu=None, sp=True)
    assert torch.equal(_kind(y), _kind(ref["out"][:, 0])) and torch.equal(_kind(state), _kind(ref["state"])) and bool((_kind(y) != 0).any())


@pytest.mark.parametrize("dtype,D,G,S,N,what,at", [
    # channels that do not fill a tile: an infinite b or c beside lanes without a channel
    (FF, 70, 1, 64, 16, "b", 20), (BF, 70, 1, 160, 8, "c", 20), (HF, 12, 2, 32, 40, "b", 5), (FF, 5, 1, 16, 5, "c", 15), (FF, 3, 1, 32, 100, "b", 31),
    # the last token of a sequence that ends inside a tile
    (FF, 8, 1, 197, 16, "dout", 196), (BF, 20, 1, 203, 6, "dout", 202), (FF, 6, 1, 205, 3, "dout", 204)])
def test_infinite_input_at_the_edge_of_a_tile(dtype, D, G, S, N, what, at):
    """What lies behind the channels or the tokens of a tile stays out of the gradients."""
    g = _gen(N + S)
    pos = lambda *s: (torch.rand(*s, generator=g) + 0.5)  # noqa: E731
    x = {k: pos(1, S, D).to(dtype).cuda() for k in ("u", "dt", "z")}
    x["dt"] = x["dt"] * -2
    x.update({k: pos(1, S, G, N).to(dtype).cuda() for k in ("b", "c")})
    x.update(a=-pos(D, N).cuda() * 0.2, d=pos(D).cuda(), dt_bias=torch.zeros(D).cuda(), initial_state=pos(1, D, N).cuda())
    dout, ds = pos(1, S, D).to(dtype).cuda(), pos(1, D, N).cuda()
    t = dout if what == "dout" else x[what]
    t[(0, at, 2) if what == "dout" else (0, at, 0, N // 2)] = float("inf")
    gr = m.mamba_scan_bwd(dout, **x, dstate=ds, dt_softplus=True)
    x["initial"] = x.pop("initial_state")
    ref = R.scan(**x, cu=None, sp=True, dout=dout, dstate=ds)
    for k, v in gr._asdict().items():
        assert torch.equal(_kind(v), _kind(ref[k])), k
    assert bool((_kind(ref["dinitial_state" if what in ("c", "dout") else "dc"]) == 1).any())


def test_norm_of_more_rows_than_one_axis_of_blocks():
    """Eight threads a row and 2^29 rows: 2^32 threads and more. The last rows as by themselves, the first as well."""
    rows, D, n = (1 << 29) + 1000, 2, 3000
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(rows, D, dtype=BF, device="cuda").normal_(generator=g)
    w = torch.tensor([0.7, -1.3], device="cuda")
    y = m.mamba_norm_fwd(x, w, activation="silu", out=torch.full_like(x, float("nan")))
    assert not bool(y.isnan().any())        # every row was written
    for part in (slice(0, n), slice(rows // 2, rows // 2 + n), slice(rows - n, rows)):
        assert _same(y[part], m.mamba_norm_fwd(x[part].clone(), w, activation="silu"))
