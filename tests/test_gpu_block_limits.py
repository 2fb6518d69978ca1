"""The gated linear recurrence and the residual addition with its norm at the limits that the header states: the bits of a call for a
part of the tensors alone."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from .test_gpu_layer import _need_gpu, _same  # noqa: F401

pytestmark = pytest.mark.gpu
BF, FF = torch.bfloat16, torch.float32


def _inputs(lead, n, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {k: new(*lead, D).to(dtype) for k in ("x", "r", "i", "z")}
    x.update(decay=new(D) - 3, r_bias=new(D), i_bias=new(D), initial_state=new(n, D))
    return x, new(*lead, D).to(dtype), new(n, D)


def _part(x, tokens, seqs, cols=slice(None)):
    f = {}
    for k, v in x.items():
        if k in ("x", "r", "i", "z", "dout"):
            f[k] = v[tokens][..., cols].contiguous()
        else:
            f[k] = (v[seqs] if v.dim() == 2 else v)[..., cols].contiguous()
    return f


def _agree(x, dout, ds, args, tokens, seqs, part_args, cols=slice(None), dinit=None):
    """dinit: the most by which dinitial_state may differ, where one call has several chunks and the other one has not."""
    a, b = m.mamba_recur_fwd(**x, **args, return_state=True), None
    p = _part({**x, "dout": dout, "dstate": ds}, tokens, seqs, cols)
    fwd = {k: v for k, v in p.items() if k not in ("dout", "dstate")}
    b = m.mamba_recur_fwd(**fwd, **part_args, return_state=True)
    assert _same(a.out[tokens][..., cols], b.out) and _same(a.state[seqs][..., cols], b.state)
    ga, gb = m.mamba_recur_bwd(dout, **x, dstate=ds, **args), m.mamba_recur_bwd(**p, **part_args)
    for k in ("dx", "dr", "di", "dz"):
        assert _same(getattr(ga, k)[tokens][..., cols], getattr(gb, k)), k
    p, q = ga.dinitial_state[seqs][..., cols], gb.dinitial_state
    assert _same(p, q) if dinit is None else bool(((p.double() - q.double()).abs() <= dinit).all())


@pytest.mark.parametrize("S", [1, 3, 130])
def test_recur_of_65535_dense_sequences(S):
    n = 65535
    x, dout, ds = _inputs((n, S), n, 6, BF, 1)
    last = slice(n - 3, n)
    _agree(x, dout, ds, {}, last, last, {})


def test_recur_of_65535_packed_sequences():
    """Lengths 0, 1, 2, 0, 1, 2, ...: the last six sequences alone are packed as a batch with the same mean."""
    n = 65535
    lens = torch.arange(n) % 3
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)
    T = int(ends[-1])
    x, dout, ds = _inputs((T,), n, 5, FF, 2)
    tail = slice(int(ends[n - 6]), T)
    # Six tokens are one chunk, whose adjoint is walked: a0 (dh0 + a1 (dh1 + a2 ds)), a <= 1; a call of several joins chunks by their products of a:
    # (a0 dh0 + a0 a1 dh1) + a0 a1 a2 ds. With two tokens at most either rounds a term up to four times: 8 * 2^-24 of the terms, |dh| <= |dout z|.
    most = (dout.double() * x["z"].double()).abs()
    terms = ds[n - 6:].double().abs() + torch.stack([most[int(a):int(b)].sum(0) for a, b in zip(ends[n - 6:], ends[n - 5:])])
    _agree(x, dout, ds, dict(cu_seqlens=ends.cuda()), tail, slice(n - 6, n), dict(cu_seqlens=(ends[n - 6:] - ends[n - 6]).cuda()), dinit=8 * 2.0 ** -24 * terms)


@pytest.mark.parametrize("S", [20, 300])
def test_recur_of_2_to_20_channels(S):
    D = 1 << 20
    x, dout, ds = _inputs((1, S), 1, D, BF, 3)
    _agree(x, dout, ds, {}, slice(None), slice(None), {}, slice(D - 70, D))


def test_recur_step_of_65535_rows():
    """Each slot of a pool comes up many times, in row order: as many calls of one row each slot."""
    n, D, slots, rounds = 65535, 10, 6000, 11
    x, _, _ = _inputs((n,), 1, D, FF, 4)
    x.pop("initial_state")
    idx = (torch.arange(n) * 7919 % slots).to(torch.int32).cuda()       # 7919 has no divisor in common with 6000: rows k, k + 6000, ... share one
    par = {k: x[k] for k in ("decay", "r_bias", "i_bias")}
    a, b = torch.zeros(slots, D, device="cuda"), torch.zeros(slots, D, device="cuda")
    out = m.mamba_recur_step(state=a, state_indices=idx, **x)
    for k in range(rounds):
        rows = slice(k * slots, min(n, (k + 1) * slots))
        one = {name: x[name][rows] for name in ("x", "r", "i", "z")}
        assert _same(out[rows], m.mamba_recur_step(state=b, state_indices=idx[rows].contiguous(), **one, **par))
    assert rounds * slots >= n and _same(a, b)


@pytest.mark.parametrize("kind", [None, torch.int8])
def test_add_norm_of_more_rows_than_one_axis_of_blocks_takes(kind):
    """32 rows a block of 256 threads, 2^32 threads an axis: 2^29 rows are on its border, some more take a second one."""
    rows, D = (1 << 29) + 1000, 1
    x, w = torch.zeros(rows, D, dtype=BF, device="cuda"), torch.full((D,), 1.5, device="cuda")
    x[-2000:] = torch.randn(2000, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    a, b = (m.mamba_add_norm_fwd(t, w, out_dtype=kind) for t in (x, x[-2000:].clone()))
    assert torch.equal(a.out[-2000:].view(torch.int8), b.out.view(torch.int8)) and not a.out[:-2000].view(torch.int8).any()
    assert kind is None or _same(a.scale[-2000:], b.scale)
    del a
    if kind is None:
        p, q = m.mamba_add_norm_bwd(x, x, w, x), m.mamba_add_norm_bwd(x[-2000:].clone(), x[-2000:].clone(), w, x[-2000:].clone())
        assert _same(p.dx[-2000:], q.dx) and not p.dx[:-2000].any()
