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
