"""Host-side checks of the layer operators (no GPU needed): the C library exports what include/mamba_layer.h
declares, the ctypes mirrors have the C layout, both the C entry points and the Python ones refuse bad
arguments before any device work."""

import ctypes
import re
import subprocess
from pathlib import Path

import pytest
import torch

import mamba_mimo_chunked_amd as m
from mamba_mimo_chunked_amd import _lib, layer

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "mamba_layer.h"


def test_library_exports_every_declared_symbol():
    decl = set(re.findall(r"^mimo_status (mamba_\w+)\s*\(", HEADER.read_text(), re.M))
    want = set(_lib.LAYER_CALLS) | {f + "_workspace_size" for f, (_, ws) in _lib.LAYER_CALLS.items() if ws}
    assert decl == want
    for name in decl:
        assert hasattr(_lib.lib(), name), name


@pytest.mark.parametrize("cls", [_lib.MambaRows] + [c for c, _ in _lib.LAYER_CALLS.values()])
def test_struct_layout_matches_c(tmp_path, cls):
    cname = re.sub(r"(?<!^)(?=[A-Z])", "_", cls.__name__).lower()
    fields = [f[0] for f in cls._fields_]
    prog = ["#include <stddef.h>", "#include <stdio.h>", '#include "mamba_layer.h"', "int main(void){",
            f'printf("%zu\\n", sizeof({cname}));']
    prog += [f'printf("%zu\\n", offsetof({cname}, {f}));' for f in fields] + ["return 0;}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(prog))
    subprocess.run(["gcc", f"-I{ROOT / 'include'}", str(src), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f in fields]


# ---------------------------------------------------------------- the C entry points
def _args(cls, **kw):
    """Arguments that pass every check but those of the device: fake aligned addresses."""
    a = cls()
    sizes = dict(n=2, S=300, D=64, W=4, G=2, N=16, slots=2, slot_stride=4096, x_stride=64, z_stride=64, dout_stride=64, rows=5, eps=1e-5)
    for f, t in cls._fields_:
        if f in sizes:
            setattr(a, f, sizes[f])
        elif t is ctypes.c_void_p and f not in ("cu_seqlens", "workspace"):
            setattr(a, f, 1 << 20)
        elif t is _lib.MambaRows:
            setattr(a, f, _lib.MambaRows(1 << 20, 64 * 300, 64))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


VALUE, TYPE, UNSUPPORTED = _lib.MIMO_ERR_VALUE, _lib.MIMO_ERR_TYPE, _lib.MIMO_ERR_UNSUPPORTED
CONV, SCAN, NORM = ("mamba_conv_fwd", "mamba_conv_bwd", "mamba_conv_step"), ("mamba_scan_fwd", "mamba_scan_bwd", "mamba_scan_step"), \
    ("mamba_norm_fwd", "mamba_norm_bwd")
BAD = [(f, kw, st) for fs, cases in (
    (CONV + SCAN, [(dict(n=0), VALUE), (dict(D=0), VALUE), (dict(dtype=3), TYPE), (dict(dtype=-1), TYPE), (dict(n=70000), UNSUPPORTED),
                   (dict(D=1 << 21), UNSUPPORTED)]),
    (CONV[:2] + SCAN[:2], [(dict(S=0), VALUE), (dict(S=(1 << 30) + 1), UNSUPPORTED)]),
    (CONV, [(dict(W=1), UNSUPPORTED), (dict(W=9), UNSUPPORTED), (dict(weight=None), VALUE)]),
    (SCAN, [(dict(N=0), VALUE), (dict(N=129), UNSUPPORTED), (dict(G=0), VALUE), (dict(G=3), VALUE), (dict(a=None), VALUE)]),
    (("mamba_conv_step", "mamba_scan_step"), [(dict(state=None), VALUE), (dict(slots=0), VALUE), (dict(indices=None, slots=1), VALUE)]),
    (("mamba_conv_fwd", "mamba_scan_fwd", "mamba_conv_step", "mamba_scan_step", "mamba_norm_fwd"), [(dict(out=None), VALUE)]),
    (("mamba_scan_bwd",), [(dict(dz=None), VALUE), (dict(z=_lib.MambaRows(None, 0, 0)), VALUE), (dict(db=None), VALUE)]),
    (NORM, [(dict(rows=0), VALUE), (dict(G=5), VALUE), (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE), (dict(silu=1), VALUE),
            (dict(dtype=7), TYPE), (dict(D=8194, G=1), UNSUPPORTED), (dict(weight=None), VALUE)]),
    (("mamba_norm_bwd",), [(dict(dz=None), VALUE), (dict(dbias=None), VALUE), (dict(z=None), VALUE)]),
) for f in fs for kw, st in cases]


@pytest.mark.parametrize("fn,kw,status", BAD)
def test_c_call_refuses(fn, kw, status):
    cls, ws = _lib.LAYER_CALLS[fn]
    L = _lib.lib()
    assert getattr(L, fn)(ctypes.byref(_args(cls, **kw)), None) == status
    assert _lib.last_error()
    assert getattr(L, fn)(None, None) == VALUE


@pytest.mark.parametrize("fn", [f for f, (_, ws) in _lib.LAYER_CALLS.items() if ws])
def test_c_call_checks_its_workspace(fn):
    cls, _ = _lib.LAYER_CALLS[fn]
    L, need = _lib.lib(), ctypes.c_size_t(0)
    a = _args(cls)
    assert getattr(L, fn + "_workspace_size")(ctypes.byref(a), ctypes.byref(need)) == _lib.MIMO_OK and need.value > 0
    assert getattr(L, fn + "_workspace_size")(ctypes.byref(a), None) == VALUE
    for ptr, size, msg in ((1 << 24, need.value - 1, "too small"), (None, need.value, "too small"), ((1 << 24) + 64, need.value, "256-byte")):
        a.workspace, a.workspace_bytes = ptr, size
        assert getattr(L, fn)(ctypes.byref(a), None) == VALUE
        assert msg in _lib.last_error()


# ---------------------------------------------------------------- the Python entry points
@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors stand in for device ones; a call that gets past the checks is an error."""
    monkeypatch.setattr(layer, "_device", lambda what, name, x: x.device)

    def reached(fn, args, device, workspace=None):
        raise AssertionError(f"{fn} was queued")
    monkeypatch.setattr(layer, "_call", reached)


def _conv(**kw):
    a = dict(x=torch.zeros(2, 6, 8), weight=torch.zeros(8, 4), bias=torch.zeros(8), initial_state=torch.zeros(2, 3, 8))
    return {**a, **kw}


def _scan(**kw):
    z = torch.zeros
    a = dict(u=z(2, 6, 8), dt=z(2, 6, 8), a=z(8, 4), b=z(2, 6, 2, 4), c=z(2, 6, 2, 4), d=z(8), z=z(2, 6, 8), dt_bias=z(8), initial_state=z(2, 8, 4))
    return {**a, **kw}


Z, I32, BF = torch.zeros, torch.int32, torch.bfloat16
PY = [
    (m.mamba_conv_fwd, _conv, [
        (dict(x=Z(2, 6, 8, dtype=torch.float64)), TypeError), (dict(x=Z(6, 8)), ValueError), (dict(x=Z(0, 6, 8)), ValueError),
        (dict(x=Z(2, 0, 8)), ValueError), (dict(weight=Z(7, 4)), ValueError), (dict(weight=Z(8, 4, dtype=BF)), TypeError),
        (dict(weight=Z(8, 1)), NotImplementedError), (dict(weight=Z(8, 9)), NotImplementedError), (dict(bias=Z(7)), ValueError),
        (dict(initial_state=Z(2, 4, 8)), ValueError), (dict(initial_state=Z(2, 3, 8, dtype=BF)), TypeError),
        (dict(activation="relu"), ValueError), (dict(cu_seqlens=Z(3, dtype=I32)), ValueError),
        (dict(x=Z(12, 8), cu_seqlens=Z(1, dtype=I32)), ValueError), (dict(x=Z(12, 8), cu_seqlens=Z(3, dtype=torch.int64)), TypeError),
        (dict(x=Z(12, 8), cu_seqlens=Z(4, dtype=I32)), ValueError), (dict(out=Z(2, 6, 7)), ValueError),
        (dict(out=Z(2, 6, 8, dtype=BF)), TypeError), (dict(out=Z(2, 8, 6).transpose(1, 2)), ValueError)]),
    (m.mamba_conv_bwd, lambda **kw: _conv(**{**dict(dout=Z(2, 6, 8)), **kw}), [
        (dict(dout=Z(2, 6, 7)), ValueError), (dict(dout=Z(2, 6, 8, dtype=BF)), TypeError), (dict(dstate=Z(2, 2, 8)), ValueError)]),
    (m.mamba_conv_step, lambda **kw: {**dict(x=Z(2, 8), state=Z(4, 3, 8), weight=Z(8, 4)), **kw}, [
        (dict(x=Z(2, 1, 8)), ValueError), (dict(x=Z(0, 8)), ValueError), (dict(state=Z(4, 4, 8)), ValueError), (dict(state=Z(1, 3, 8)), ValueError),
        (dict(state=Z(4, 3, 8, dtype=BF)), TypeError), (dict(state=Z(4, 8, 3).transpose(1, 2)), ValueError),
        (dict(state=Z(1, 3, 8).expand(4, 3, 8)), ValueError), (dict(state_indices=Z(3, dtype=I32)), ValueError),
        (dict(state_indices=Z(2, dtype=torch.int64)), TypeError), (dict(state=Z(0, 3, 8), state_indices=Z(2, dtype=I32)), ValueError)]),
    (m.mamba_scan_fwd, _scan, [
        (dict(u=Z(2, 6, 8, dtype=torch.int32)), TypeError), (dict(dt=Z(2, 6, 8, dtype=BF)), TypeError), (dict(dt=Z(2, 6, 7)), ValueError),
        (dict(a=Z(7, 4)), ValueError), (dict(a=Z(8, 4, dtype=BF)), TypeError), (dict(a=Z(8, 129), b=Z(2, 6, 2, 129), c=Z(2, 6, 2, 129)), NotImplementedError),
        (dict(b=Z(2, 6, 2, 5)), ValueError), (dict(b=Z(2, 6, 4)), ValueError), (dict(b=Z(2, 6, 3, 4), c=Z(2, 6, 3, 4)), ValueError),
        (dict(c=Z(2, 6, 1, 4)), ValueError), (dict(d=Z(4)), ValueError), (dict(z=Z(2, 6, 4)), ValueError), (dict(dt_bias=Z(8, dtype=BF)), TypeError),
        (dict(initial_state=Z(2, 4, 8)), ValueError), (dict(initial_state=Z(2, 8, 4, dtype=BF)), TypeError), (dict(out=Z(12, 8)), ValueError),
        (dict(cu_seqlens=Z(3, dtype=I32)), ValueError)]),
    (m.mamba_scan_bwd, lambda **kw: _scan(**{**dict(dout=Z(2, 6, 8)), **kw}), [
        (dict(dout=Z(2, 5, 8)), ValueError), (dict(dstate=Z(2, 8, 5)), ValueError), (dict(dstate=Z(2, 8, 4, dtype=BF)), TypeError)]),
    (m.mamba_scan_step, lambda **kw: {**dict(u=Z(2, 8), dt=Z(2, 8), state=Z(4, 8, 4), a=Z(8, 4), b=Z(2, 2, 4), c=Z(2, 2, 4)), **kw}, [
        (dict(u=Z(8)), ValueError), (dict(b=Z(2, 4)), ValueError), (dict(state=Z(4, 4, 8)), ValueError), (dict(state=Z(4, 8, 4, dtype=BF)), TypeError),
        (dict(state=Z(4, 4, 8).transpose(1, 2)), ValueError), (dict(state=Z(1, 8, 4)), ValueError), (dict(state_indices=Z(2, 1, dtype=I32)), ValueError)]),
    (m.mamba_norm_fwd, lambda **kw: {**dict(x=Z(2, 3, 8), weight=Z(8)), **kw}, [
        (dict(x=Z(2, 3, 8, dtype=torch.float64)), TypeError), (dict(x=Z(0, 8)), ValueError), (dict(weight=Z(7)), ValueError),
        (dict(bias=Z(8, dtype=BF)), TypeError), (dict(z=Z(2, 8)), ValueError), (dict(groups=3), ValueError), (dict(groups=0), ValueError),
        (dict(groups=True), ValueError), (dict(eps=-1e-5), ValueError), (dict(eps=float("nan")), ValueError), (dict(gate="between"), ValueError),
        (dict(z=Z(2, 3, 8), activation="silu"), ValueError), (dict(x=Z(1, 8193), weight=Z(8193)), NotImplementedError), (dict(out=Z(6, 8)), ValueError)]),
    (m.mamba_norm_bwd, lambda **kw: {**dict(dout=Z(2, 3, 8), x=Z(2, 3, 8), weight=Z(8)), **kw}, [
        (dict(dout=Z(3, 8)), ValueError), (dict(dout=Z(2, 3, 8, dtype=BF)), TypeError)]),
]


@pytest.mark.parametrize("fn,make,kw,exc", [(f, mk, kw, e) for f, mk, cases in PY for kw, e in cases])
def test_python_call_refuses(on_cpu, fn, make, kw, exc):
    with pytest.raises(exc):
        fn(**make(**kw))


@pytest.mark.parametrize("fn,make", [(f, mk) for f, mk, _ in PY])
def test_good_arguments_pass_the_checks(on_cpu, fn, make):
    with pytest.raises(AssertionError, match="was queued"):
        fn(**make())


def test_outputs_may_not_overlap_inputs(on_cpu):
    x, w, out = Z(1, 6, 8), Z(8, 4), torch.zeros(2, 6, 8)
    with pytest.raises(ValueError, match="overlap x"):
        m.mamba_conv_fwd(x, w, out=x)
    with pytest.raises(ValueError, match="overlap x"):
        m.mamba_norm_fwd(x, Z(8), out=x)
    with pytest.raises(ValueError, match="overlap u"):
        a = _scan(u=out)
        m.mamba_scan_fwd(**a, out=out)
    bias = Z(48)
    with pytest.raises(ValueError, match="overlap bias"):
        m.mamba_conv_fwd(Z(1, 1, 48), Z(48, 4), bias, out=bias.view(1, 1, 48))
    with pytest.raises(ValueError, match="overlap weight"):
        m.mamba_norm_fwd(Z(1, 48), bias, out=bias.view(1, 48))
    pool = Z(3, 8, 4)
    with pytest.raises(ValueError, match="overlap"):
        m.mamba_scan_step(pool.view(-1)[:16].view(2, 8), Z(2, 8), pool, Z(8, 4), Z(2, 2, 4), Z(2, 2, 4))


@pytest.mark.parametrize("fn,make", [(f, mk) for f, mk, _ in PY])
def test_cpu_tensors_are_refused(fn, make):
    with pytest.raises(ValueError, match="GPU"):
        fn(**make())
