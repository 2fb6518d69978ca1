"""Host-side checks of the gated linear recurrence and the residual addition's norm (no GPU needed): the C entry points and the
Python ones refuse bad arguments before any device work, and nothing that is written may lie over what is read."""

import ctypes

import pytest
import torch

import mamba_mimo_chunked_amd as m
from mamba_mimo_chunked_amd import _lib

from .test_layer_boundary import TYPE, UNSUPPORTED, VALUE, _args, on_cpu  # noqa: F401
from .test_layer_limits import _query

RECUR, ADD = ("mamba_recur_fwd", "mamba_recur_bwd", "mamba_recur_step"), ("mamba_add_norm_fwd", "mamba_add_norm_bwd")
NONE = _lib.MambaRows(None, 0, 0)
BAD = [(f, kw, st) for fs, cases in (
    (RECUR, [(dict(n=0), VALUE), (dict(D=0), VALUE), (dict(dtype=3), TYPE), (dict(dtype=-1), TYPE), (dict(n=70000), UNSUPPORTED),
             (dict(D=1 << 21), UNSUPPORTED), (dict(rate=-1.0), VALUE), (dict(rate=float("nan")), VALUE), (dict(rate=float("inf")), VALUE),
             (dict(x=NONE), VALUE), (dict(r=NONE), VALUE), (dict(i=NONE), VALUE), (dict(decay=None), VALUE)]),
    (RECUR[:2], [(dict(S=0), VALUE), (dict(S=(1 << 30) + 1), UNSUPPORTED), (dict(r=_lib.MambaRows(1 << 20, 0, (1 << 26) + 1)), UNSUPPORTED),
                 (dict(z=_lib.MambaRows(1 << 20, 0, -64)), UNSUPPORTED)]),
    (("mamba_recur_fwd", "mamba_recur_step"), [(dict(out=None), VALUE)]),
    (("mamba_recur_step",), [(dict(state=None), VALUE), (dict(slots=0), VALUE), (dict(indices=None, slots=1), VALUE)]),
    (("mamba_recur_bwd",), [(dict(dout=NONE), VALUE), (dict(dz=None), VALUE), (dict(z=NONE), VALUE), (dict(dr_bias=None), VALUE), (dict(i_bias=None), VALUE),
                            (dict(dx=None), VALUE), (dict(ddecay=None), VALUE)]),
    (ADD, [(dict(rows=0), VALUE), (dict(D=0), VALUE), (dict(D=16385), UNSUPPORTED), (dict(rows=(1 << 31) + 1), UNSUPPORTED), (dict(dtype=3), TYPE),
           (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(drop=-1), VALUE), (dict(drop=65536), VALUE), (dict(drop=9, seed=None), VALUE),
           (dict(weight=None), VALUE), (dict(x=None, sum=None, dout=None), VALUE)]),
    (ADD[:1], [(dict(out=None), VALUE), (dict(out_kind=3), TYPE), (dict(out_kind=-1), TYPE), (dict(out_kind=1, block=33), VALUE), (dict(out_kind=1, block=-32), VALUE),
               (dict(block=32), VALUE), (dict(out_kind=2, scale=None), VALUE), (dict(sum=None), VALUE), (dict(sum=None, residual=None, wide=1), VALUE),
               (dict(sum=None, residual=None, drop=5), VALUE)]),
    (ADD[1:], [(dict(dx=None), VALUE), (dict(dweight=None), VALUE)]),
) for f in fs for kw, st in cases]


@pytest.mark.parametrize("fn,kw,status", BAD)
def test_c_call_refuses(fn, kw, status):
    cls, ws = _lib.LAYER_CALLS[fn]
    fields = {f for f, _ in cls._fields_}
    assert getattr(_lib.lib(), fn)(ctypes.byref(_args(cls, **{k: v for k, v in kw.items() if k in fields})), None) == status
    assert _lib.last_error()


@pytest.mark.parametrize("fn", ["mamba_recur_fwd", "mamba_recur_bwd"])
def test_more_threads_than_a_grid_holds(fn):
    """65535 sequences of 2^20 tokens: refused by the query already. A long narrow sequence is taken."""
    assert _query(fn, n=65535, S=1 << 20, D=2)[0] == UNSUPPORTED
    assert _query(fn, n=1, S=1 << 26, D=64)[0] == _lib.MIMO_OK


@pytest.mark.parametrize("n,S,D,packed", [(4, 4096, 2048, False), (1, 128, 64, False), (1, 129, 64, False), (5, 64, 10, False), (5, 65, 10, False), (9, 16, 70, False),
                                          (9, 17, 70, False), (1, 1, 1, False), (2000, 16000, 2048, True), (160, 16000, 1025, True), (1, 16, 8, True), (1, 5, 8, True),
                                          (3, 64, 8, True), (2, 200, 33, True), (70, 4, 8, True)])
def test_workspace_of_the_recurrence_is_what_the_header_states(n, S, D, packed):
    cu = 1 << 20 if packed else None
    short = packed and S // n < 64
    for fn, C in (("mamba_recur_fwd", 32 if short else 64 if packed else 128), ("mamba_recur_bwd", 16 if short else 32 if packed else 64)):
        chunks = S // C + n + 1 if packed else n * -(-S // C)
        if fn.endswith("fwd"):
            want, slack = (8 * D * (chunks + chunks // (C // 4)), 8 * D + 256 * (-(-D // 64) + 3)) if S > C else (0, 0)
        else:
            want, slack = 12 * D * chunks * (2 if S > C else 1), 4 * 256
        status, got = _query(fn, n=n, S=S, D=D, cu_seqlens=cu)
        assert status == _lib.MIMO_OK and want <= got <= want + slack, (fn, want, got)


Z, F16, I32, U8 = torch.zeros, torch.float16, torch.int32, torch.uint8


def _recur(**kw):
    a = dict(x=Z(2, 6, 8), r=Z(2, 6, 8), i=Z(2, 6, 8), decay=Z(8), r_bias=Z(8), i_bias=Z(8), z=Z(2, 6, 8), initial_state=Z(2, 8))
    return {**a, **kw}


def _step(**kw):
    a = dict(x=Z(2, 8), r=Z(2, 8), i=Z(2, 8), state=Z(4, 8), decay=Z(8), r_bias=Z(8), i_bias=Z(8), z=Z(2, 8), state_indices=Z(2, dtype=I32))
    return {**a, **kw}


def _add(**kw):
    return {**dict(x=Z(3, 8), weight=Z(8), residual=Z(3, 8)), **kw}


def _addb(**kw):
    return {**dict(dout=Z(3, 8), sum=Z(3, 8), weight=Z(8), dsum=Z(3, 8)), **kw}


REFUSED = [
    (m.mamba_recur_fwd, _recur, ValueError, [dict(r=None), dict(i=None), dict(decay=None), dict(x=Z(6, 8)), dict(x=Z(2, 0, 8), r=Z(2, 0, 8)), dict(r=Z(2, 6, 7)),
                                             dict(i=Z(2, 5, 8)), dict(z=Z(1, 6, 8)), dict(decay=Z(7)), dict(r_bias=Z(8, 1)), dict(initial_state=Z(2, 8, 1)),
                                             dict(rate=-0.5), dict(rate=float("nan")), dict(rate=float("inf")), dict(cu_seqlens=Z(3, dtype=I32)), dict(out=Z(2, 6, 9)),
                                             dict(out=Z(2, 8, 6).transpose(1, 2))]),
    (m.mamba_recur_fwd, _recur, TypeError, [dict(x=Z(2, 6, 8, dtype=torch.float64)), dict(r=Z(2, 6, 8, dtype=F16)), dict(decay=Z(8, dtype=F16)),
                                            dict(initial_state=Z(2, 8, dtype=F16)), dict(out=Z(2, 6, 8, dtype=F16))]),
    (m.mamba_recur_bwd, lambda **kw: _recur(**{"dout": Z(2, 6, 8), **kw}), ValueError, [dict(dout=None), dict(dout=Z(2, 6, 7)), dict(dstate=Z(2, 9)), dict(rate=-1)]),
    (m.mamba_recur_bwd, lambda **kw: _recur(**{"dout": Z(2, 6, 8), **kw}), TypeError, [dict(dout=Z(2, 6, 8, dtype=F16)), dict(dstate=Z(2, 8, dtype=F16))]),
    (m.mamba_recur_step, _step, ValueError, [dict(x=Z(2, 1, 8)), dict(x=Z(0, 8)), dict(state=None), dict(state=Z(4, 9)), dict(state=Z(4, 1, 8)), dict(state=Z(4)),
                                             dict(state=Z(0, 8)), dict(state=Z(1, 8), state_indices=None), dict(state=Z(4, 16)[:, ::2]), dict(state=Z(8).expand(4, 8)),
                                             dict(state_indices=Z(3, dtype=I32)), dict(rate=float("inf"))]),
    (m.mamba_recur_step, _step, TypeError, [dict(state=Z(4, 8, dtype=F16)), dict(state_indices=Z(2, dtype=torch.int64))]),
    (m.mamba_add_norm_fwd, _add, ValueError, [dict(weight=None), dict(x=Z(0, 8), residual=None), dict(weight=Z(7)), dict(residual=Z(2, 8)), dict(eps=-1e-5),
                                              dict(eps=float("nan")), dict(dropout=1.0), dict(dropout=-0.1), dict(dropout=float("nan")), dict(dropout=0.1),
                                              dict(dropout=0.1, seed=Z(3, dtype=torch.int64)), dict(block=32), dict(block=33, out_dtype=torch.int8),
                                              dict(block=0, out_dtype=torch.int8), dict(out=Z(3, 9)), dict(out=Z(8, 3).t())]),
    (m.mamba_add_norm_fwd, _add, TypeError, [dict(x=Z(3, 8, dtype=torch.float64)), dict(weight=Z(8, dtype=F16)), dict(residual=Z(3, 8, dtype=F16)), dict(sum_dtype=F16),
                                             dict(x=Z(3, 8, dtype=F16), sum_dtype=F16), dict(residual=None, sum_dtype=torch.bfloat16),
                                             dict(out_dtype=torch.uint8), dict(out_dtype=F16), dict(dropout=0.1, seed=Z(2, dtype=I32)), dict(out=Z(3, 8, dtype=F16))]),
    (m.mamba_add_norm_fwd, _add, NotImplementedError, [dict(x=Z(1, 16385), weight=Z(16385), residual=None)]),
    (m.mamba_add_norm_bwd, _addb, ValueError, [dict(sum=None), dict(weight=None), dict(sum=Z(3, 7)), dict(dsum=Z(2, 8)), dict(dropout=0.1), dict(eps=-1)]),
    (m.mamba_add_norm_bwd, _addb, TypeError, [dict(sum=Z(3, 8, dtype=F16)), dict(dsum=Z(3, 8, dtype=F16)), dict(dout=Z(3, 8, dtype=torch.int8))]),
]


@pytest.mark.parametrize("fn,make,err,kw", [(f, mk, e, kw) for f, mk, e, kws in REFUSED for kw in kws])
def test_python_call_refuses(on_cpu, fn, make, err, kw):  # noqa: F811
    with pytest.raises(err):
        fn(**make(**kw))


def test_first_tensor_is_required_and_on_the_gpu():
    for fn, make, name in ((m.mamba_recur_fwd, _recur, "x"), (m.mamba_recur_step, _step, "x"), (m.mamba_add_norm_fwd, _add, "x"), (m.mamba_add_norm_bwd, _addb, "dout")):
        with pytest.raises(ValueError, match=f"{name} is required"):
            fn(**make(**{name: None}))
        with pytest.raises(ValueError, match="requires GPU"):
            fn(**make())


def test_good_calls_pass(on_cpu):  # noqa: F811
    for fn, a in ((m.mamba_recur_fwd, _recur()), (m.mamba_recur_bwd, _recur(dout=Z(2, 6, 8))), (m.mamba_recur_step, _step()), (m.mamba_recur_step, _step(state=Z(4, 9)[:, :8])),
                  (m.mamba_add_norm_fwd, _add()), (m.mamba_add_norm_fwd, _add(out_dtype=torch.float8_e4m3fn, block=32)), (m.mamba_add_norm_fwd, _add(x=Z(3, 8, dtype=F16))),
                  (m.mamba_add_norm_fwd, _add(dropout=1e-9)), (m.mamba_add_norm_bwd, _addb()), (m.mamba_recur_fwd, _recur(rate=0))):
        with pytest.raises(AssertionError, match="was queued"):
            fn(**a)


def _over(x):
    return x.view(U8).view(-1)


@pytest.mark.parametrize("name", ["x", "r", "i", "decay", "r_bias", "i_bias", "z", "initial_state", "dout", "dstate", "out"])
def test_workspace_of_the_recurrence(on_cpu, name):  # noqa: F811
    more = {"dout": Z(2, 6, 8), "dstate": Z(2, 8)} if name in ("dout", "dstate") else {"out": Z(2, 6, 8)} if name == "out" else {}
    a = _recur(**more)
    with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
        (m.mamba_recur_bwd if "dout" in a else m.mamba_recur_fwd)(**a, workspace=_over(a[name]))


@pytest.mark.parametrize("name", ["x", "r", "i", "z", "initial_state"])
def test_output_of_the_recurrence(on_cpu, name):  # noqa: F811
    buf = Z(96)
    over = buf.view(2, 6, 8) if name != "initial_state" else buf[16:32].view(2, 8)
    with pytest.raises(ValueError, match=f"out must not overlap {name}"):
        m.mamba_recur_fwd(**_recur(**{name: over}), out=buf.view(2, 6, 8))


@pytest.mark.parametrize("name", ["x", "r", "i", "z"])
def test_state_of_the_recurrence(on_cpu, name):  # noqa: F811
    buf = Z(32)
    with pytest.raises(ValueError, match=f"state must not overlap {name}"):
        m.mamba_recur_step(**_step(state=buf.view(4, 8), **{name: buf[8:24].view(2, 8)}))


def test_overlaps_of_the_addition(on_cpu):  # noqa: F811
    for name in ("x", "residual"):
        a = _add()
        with pytest.raises(ValueError, match=f"out must not overlap {name}"):
            m.mamba_add_norm_fwd(**a, out=a[name])
    for name in ("dout", "sum", "dsum", "weight"):
        a = _addb()
        with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
            m.mamba_add_norm_bwd(**a, workspace=_over(a[name]))
    a, seed = _addb(), Z(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="workspace must not overlap seed"):
        m.mamba_add_norm_bwd(**a, dropout=0.1, seed=seed, workspace=_over(seed))


def test_output_over_the_sum_that_is_x(on_cpu):  # noqa: F811
    """Where nothing is added the sum is x itself, whose rows are copied for the call if their strides need it."""
    buf = Z(96)
    x = buf.view(3, 4, 8)[:, :3]
    with pytest.raises(ValueError, match="out must not overlap x"):
        m.mamba_add_norm_fwd(x, Z(8), out=buf[:72].view(3, 3, 8))
