"""The layer operators around the scan: the short causal convolution ``mamba_conv_*``, the selective
scan ``mamba_scan_*`` with a decay for each channel and state, and the gated group norm
``mamba_norm_*``, each as a forward call, a backward call that returns the gradients, and (where there
is a state) a step of one token.

Data tensors share one dtype: bfloat16, float16 or float32. Parameters, the scan's state and their
gradients are float32; so is all arithmetic, rounded once when stored. Sequences are a dense batch
[B, S, ...] or packed along one token axis [T, ...] with ``cu_seqlens`` [n + 1] (int32, on the device:
0, then each sequence's end, not decreasing, at most T; its values are not checked, and sequences may
be empty). Token and batch strides are free as long as the inner axes are dense; other layouts are
copied. What a call writes (a given output or workspace, a pool of states) must not overlap what it
reads. Calls are asynchronous on the current HIP stream of the tensors' device. Sums run in a fixed
order: equal inputs give equal bits. Limits, infinite inputs and the size of workspaces:
``include/mamba_layer.h``.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _BWD2_DTYPES as _DTYPES
from .api import _check_output, _check_tensor, _is_gfx950, _raise, _workspace

__all__ = ["MambaConvOutputs", "MambaConvGrads", "MambaScanOutputs", "MambaScanGrads", "MambaNormGrads", "mamba_conv_fwd",
           "mamba_conv_bwd", "mamba_conv_step", "mamba_scan_fwd", "mamba_scan_bwd", "mamba_scan_step", "mamba_norm_fwd",
           "mamba_norm_bwd"]

Tensor = torch.Tensor
_F32 = torch.float32


class MambaConvOutputs(NamedTuple):
    out: Tensor
    state: Optional[Tensor]


class MambaConvGrads(NamedTuple):
    dx: Tensor
    dweight: Tensor
    dbias: Optional[Tensor]
    dinitial_state: Optional[Tensor]


class MambaScanOutputs(NamedTuple):
    out: Tensor
    state: Optional[Tensor]


class MambaScanGrads(NamedTuple):
    du: Tensor
    ddt: Tensor
    da: Tensor
    db: Tensor
    dc: Tensor
    dd: Optional[Tensor]
    dz: Optional[Tensor]
    ddt_bias: Optional[Tensor]
    dinitial_state: Optional[Tensor]


class MambaNormGrads(NamedTuple):
    dx: Tensor
    dweight: Tensor
    dbias: Optional[Tensor]
    dz: Optional[Tensor]


# ---------------------------------------------------------------- checks
# A step of one token takes the GPU about three microseconds, so what happens here is kept short: a tensor is
# looked at once, its pointer taken once, and the arguments packed as bytes instead of ctypes fields.
def _data_dtype(name, x):
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must use torch.bfloat16, torch.float16 or torch.float32, got {x.dtype}")
    return code


_READY = set()   # devices that passed the checks


def _device(what, name, x):
    """The device of the first tensor; every other one has to be there too."""
    if x is None:
        raise ValueError(f"{name} is required")
    dev = x.device
    if dev in _READY:
        return dev
    if dev.type != "cuda":
        raise ValueError(f"{what} requires GPU (HIP) tensors, got {name} on {dev}")
    if not _is_gfx950(dev.index if dev.index is not None else torch.cuda.current_device()):
        raise NotImplementedError(f"{what} supports gfx950 (MI355X) devices only")
    _READY.add(dev)
    return dev


def _required(**tensors):
    for name, x in tensors.items():
        if x is None:
            raise ValueError(f"{name} is required")


def _fits(name, x, shape, dtype, device):
    """_check_tensor, without its cost where all is well."""
    if x.shape != shape or x.dtype != dtype or x.device != device:
        _check_tensor(name, x, shape, dtype, device)


def _param(name, x, shape, dtype, device):
    """A tensor that has to be dense (None stays None): checked, a copy where it is not dense. The caller
    keeps it until the call is queued."""
    if x is None:
        return None
    if x.shape != shape or x.dtype != dtype or x.device != device:
        _check_tensor(name, x, shape, dtype, device)
    return x if x.is_contiguous() else x.contiguous()


def _data(name, x, shape, dtype, device, inner=1):
    """A tensor whose last ``inner`` axes have to be dense: checked, a copy where they are not."""
    if x is None:
        return None
    if x.shape != shape or x.dtype != dtype or x.device != device:
        _check_tensor(name, x, shape, dtype, device)
    return x if x.is_contiguous() else _dense_inner(x, inner)


def _dense_inner(x, inner):
    """x as it is if its last ``inner`` axes are dense, else a contiguous copy."""
    if x.is_contiguous():
        return x
    step = 1
    for k in range(1, inner + 1):
        if x.shape[-k] != 1 and x.stride(-k) != step:
            return x.contiguous()
        step *= x.shape[-k]
    return x


def _sequences(name, x, cu_seqlens, inner):
    """(n, S, leading shape): a dense batch [B, S, ...] or, with cu_seqlens, tokens [T, ...]."""
    shape = tuple(x.shape)
    if cu_seqlens is None:
        if len(shape) != 2 + inner:
            raise ValueError(f"{name} must have {2 + inner} axes (batch, tokens, ...), got shape {list(shape)}")
        n, S = shape[:2]
        lead = (n, S)
    else:
        if len(shape) != 1 + inner:
            raise ValueError(f"{name} must have {1 + inner} axes (tokens, ...) with cu_seqlens, got shape {list(shape)}")
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must have shape [n + 1] with at least one sequence")
        n, S = cu_seqlens.shape[0] - 1, shape[0]
        lead = (S,)
    if 0 in shape:
        raise ValueError(f"{name} must not be empty, got shape {list(shape)}")
    return n, S, lead


def _cu(cu_seqlens, device):
    return None if cu_seqlens is None else _param("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, device)


_NO_ROWS = (0, 0, 0)


def _rows(x, packed):
    """The mamba_rows fields of a tensor whose inner axes are dense (None: no tensor)."""
    if x is None:
        return _NO_ROWS
    return (x.data_ptr(), 0, x.stride(0)) if packed else (x.data_ptr(), x.stride(0), x.stride(1))


def _ptr(x):
    return 0 if x is None else x.data_ptr()


def _span(x):
    """First and last byte (exclusive) that a tensor's elements lie in."""
    lo = x.data_ptr()
    if x.is_contiguous():
        return lo, lo + x.nbytes
    return lo, lo + (sum((s - 1) * st for s, st in zip(x.shape, x.stride())) + 1) * x.element_size()


def _apart(name, written, /, **others):
    """A tensor that is written must not lie over one that is read. One that starts where its storage starts can only
    be met by tensors that start inside it."""
    lo, hi = _span(written)
    first = written.untyped_storage().data_ptr() == lo
    for other, x in others.items():
        if x is not None:
            p = x.data_ptr()
            if p < hi and (p >= lo or (not first and _span(x)[1] > lo)):
                raise ValueError(f"{name} must not overlap {other}")


def _new_like(x):
    """A dense tensor of x's shape, type and device."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _out(out, like, /, **inputs):
    """The output: a new tensor, or the caller's."""
    if out is None:
        return _new_like(like)
    _check_output("out", out, like.shape, like.dtype, like.device)
    _apart("out", out, **inputs)
    return out


_QUEUE = {}   # entry point -> (C function, its workspace query or None, packer of the argument struct)


def _call(fn, values, device, workspace=None):
    """Queue one library call on the device's current stream. ``values``: the fields of its argument struct in
    order, without the workspace, which is added where the call has one."""
    entry = _QUEUE.get(fn)
    if entry is None:
        L = _lib.lib()
        cls, ws = _lib.LAYER_CALLS[fn]
        entry = _QUEUE[fn] = (getattr(L, fn), getattr(L, fn + "_workspace_size") if ws else None, _lib.packer(cls))
    call, query, pack = entry
    if query is not None:
        need = ctypes.c_size_t(0)
        st = query(pack(*values, 0, 0), ctypes.byref(need))
        if st != _lib.MIMO_OK:
            _raise(st)
        workspace = _workspace(workspace, need.value, device)
        values = (*values, 0, 0) if workspace is None else (*values, workspace.data_ptr(), workspace.numel())
    args, stream = pack(*values), torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() == device.index:
        st = call(args, stream)
    else:
        with torch.cuda.device(device):
            st = call(args, stream)
    if st != _lib.MIMO_OK:
        _raise(st)


# ---------------------------------------------------------------- short causal convolution
def _activation(activation):
    if activation not in (None, "silu"):
        raise ValueError("activation must be None or 'silu'")
    return int(activation == "silu")


def _check_filter(weight, bias, D, device):
    if weight is None:
        _required(weight=weight)
    shape = weight.shape
    if len(shape) != 2 or shape[0] != D:
        raise ValueError(f"weight must have shape [{D}, taps], got {list(shape)}")
    W = shape[1]
    if weight.dtype != _F32 or weight.device != device:
        _check_tensor("weight", weight, shape, _F32, device)
    if not 2 <= W <= 8:
        raise NotImplementedError(f"mamba_conv supports 2 to 8 taps, got {W}")
    return W, weight if weight.is_contiguous() else weight.contiguous(), _param("bias", bias, (D,), _F32, device)


def mamba_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, *, activation: Optional[str] = None,
                   return_state: bool = False, out: Optional[Tensor] = None) -> MambaConvOutputs:
    """Short causal convolution, one filter of W = 2..8 taps per channel: with e the sequence behind its
    W - 1 rows of state (zeros without ``initial_state``), ``out[t] = act(bias + sum_k weight[:, k] e[t + k])``,
    act the identity or SiLU.

    x, out [B, S, D] or packed [T, D]; weight [D, W] and bias [D] float32; initial_state and the returned
    ``state`` (with ``return_state``; the last W - 1 rows of e) [n, W - 1, D] in x's dtype, newest last, as
    ``mamba_conv_step`` takes them. Tokens behind the last sequence: rows of ``out`` are left as they
    were when the caller gives it, else zero."""
    dev = _device("mamba_conv_fwd", "x", x)
    code = _data_dtype("x", x)
    silu = _activation(activation)
    n, S, lead = _sequences("x", x, cu_seqlens, 1)
    D = x.shape[-1]
    W, weight, bias = _check_filter(weight, bias, D, dev)
    initial_state = _param("initial_state", initial_state, (n, W - 1, D), x.dtype, dev)
    cu, x = _cu(cu_seqlens, dev), _dense_inner(x, 1)
    res = _out(out, x, x=x, weight=weight, bias=bias, initial_state=initial_state, cu_seqlens=cu)
    state = x.new_empty((n, W - 1, D)) if return_state else None
    _call("mamba_conv_fwd", (n, S, D, W, code, silu, int(out is None), _ptr(cu), *_rows(x, cu is not None), _ptr(weight),
                             _ptr(bias), _ptr(initial_state), _ptr(res), _ptr(state)), dev)
    return MambaConvOutputs(res, state)


def mamba_conv_bwd(dout, x, weight, bias=None, initial_state=None, dstate=None, cu_seqlens=None, *,
                   activation: Optional[str] = None, workspace: Optional[Tensor] = None) -> MambaConvGrads:
    """Gradients of ``sum(out * dout) + sum(state * dstate)`` for the arguments of ``mamba_conv_fwd``: dx and
    dinitial_state in x's dtype, dweight and dbias float32; dbias and dinitial_state are None without the
    input. dout like x, dstate like initial_state. dx is zero behind the last sequence."""
    dev = _device("mamba_conv_bwd", "x", x)
    code = _data_dtype("x", x)
    silu = _activation(activation)
    n, S, lead = _sequences("x", x, cu_seqlens, 1)
    D = x.shape[-1]
    W, weight, bias = _check_filter(weight, bias, D, dev)
    if dout is None:
        _required(dout=dout)
    dout = _data("dout", dout, x.shape, x.dtype, dev)
    initial_state = _param("initial_state", initial_state, (n, W - 1, D), x.dtype, dev)
    dstate = _param("dstate", dstate, (n, W - 1, D), x.dtype, dev)
    cu, x = _cu(cu_seqlens, dev), _dense_inner(x, 1)
    dx, dweight = _new_like(x), torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    dinit = None if initial_state is None else torch.empty_like(initial_state)
    if workspace is not None:
        _apart("workspace", workspace, dout=dout, x=x, weight=weight, bias=bias, initial_state=initial_state, dstate=dstate, cu_seqlens=cu)
    packed = cu is not None
    _call("mamba_conv_bwd", (n, S, D, W, code, silu, 0, _ptr(cu), *_rows(dout, packed), *_rows(x, packed), _ptr(weight), _ptr(bias),
                             _ptr(initial_state), _ptr(dstate), _ptr(dx), _ptr(dweight), _ptr(dbias), _ptr(dinit)), dev, workspace)
    return MambaConvGrads(dx, dweight, dbias, dinit)


def _check_pool(state, inner, dtype, indices, n, device):
    """A pool of states [slots, ...]: dense inside a slot, slots that do not overlap, updated in place."""
    if state is None:
        _required(state=state)
    shape = state.shape
    if len(shape) != 3 or shape[1] != inner[0] or shape[2] != inner[1]:
        raise ValueError(f"state must have shape [slots, {', '.join(map(str, inner))}], got {list(shape)}")
    slots, size = shape[0], inner[0] * inner[1]
    if state.dtype != dtype or state.device != device:
        _check_tensor("state", state, shape, dtype, device)
    if slots < 1:
        raise ValueError("state must have at least one slot")
    stride = size
    if not state.is_contiguous():
        if (inner[1] != 1 and state.stride(2) != 1) or (inner[0] != 1 and state.stride(1) != inner[1]):
            raise ValueError("state must be dense inside a slot: it is updated in place")
        stride = state.stride(0) if slots > 1 else size
        if stride < size:
            raise ValueError("the slots of state must not overlap")
    if indices is not None:
        indices = _param("state_indices", indices, (n,), torch.int32, device)
    elif slots < n:
        raise ValueError(f"state has {slots} slots for {n} rows: without state_indices each row needs its own")
    return slots, stride, indices


def mamba_conv_step(x, state, weight, bias=None, state_indices=None, *, activation: Optional[str] = None,
                    out: Optional[Tensor] = None) -> Tensor:
    """One token of ``mamba_conv_fwd`` for each of n rows: x, out [n, D]; ``state`` [slots, W - 1, D] in x's
    dtype is updated in place. Row i uses slot ``state_indices[i]`` (int32; i without it). A row whose index
    is outside [0, slots) is skipped and its output is zero; rows with the same index are taken in row
    order, as consecutive tokens of one sequence."""
    dev = _device("mamba_conv_step", "x", x)
    code = _data_dtype("x", x)
    silu = _activation(activation)
    shape = x.shape
    if len(shape) != 2 or 0 in shape:
        raise ValueError(f"x must have shape [n, D] and not be empty, got {list(shape)}")
    n, D = shape
    W, weight, bias = _check_filter(weight, bias, D, dev)
    slots, stride, idx = _check_pool(state, (W - 1, D), x.dtype, state_indices, n, dev)
    x = _dense_inner(x, 1)
    _apart("state", state, x=x, weight=weight, bias=bias, state_indices=idx)
    res = _out(out, x, x=x, state=state, weight=weight, bias=bias, state_indices=idx)
    _call("mamba_conv_step", (n, D, slots, stride, x.stride(0), W, code, silu, 0, x.data_ptr(), state.data_ptr(), weight.data_ptr(),
                              _ptr(bias), _ptr(idx), res.data_ptr()), dev)
    return res


# ---------------------------------------------------------------- selective scan
def _check_scan(u, dt, a, b, c, d, z, dt_bias, lead, dev):
    """Sizes and the tensors with dense inner axes, parameters contiguous."""
    if dt is None or a is None or b is None or c is None:
        _required(dt=dt, a=a, b=b, c=c)
    rows, dtype, ashape, shape = u.shape, u.dtype, a.shape, b.shape
    D = rows[-1]
    if len(ashape) != 2 or ashape[0] != D:
        raise ValueError(f"a must have shape [{D}, N], got {list(ashape)}")
    N = ashape[1]
    if shape[:-2] != lead or len(shape) < 2 or shape[-1] != N:
        raise ValueError(f"b must have shape {[*lead, 'G', N]}, got {list(shape)}")
    G = shape[-2]
    if G < 1 or N < 1 or D % G:
        raise ValueError(f"the {D} channels must be divisible by the {G} groups of b and c, and a must have states")
    if N > 128:
        raise NotImplementedError(f"mamba_scan supports at most 128 states, got {N}")
    data = (_dense_inner(u, 1), _data("dt", dt, rows, dtype, dev), _data("b", b, shape, dtype, dev, 2), _data("c", c, shape, dtype, dev, 2),
            _data("z", z, rows, dtype, dev))
    return D, G, N, data, (_param("a", a, ashape, _F32, dev), _param("d", d, (D,), _F32, dev), _param("dt_bias", dt_bias, (D,), _F32, dev))


def mamba_scan_fwd(u, dt, a, b, c, d=None, z=None, dt_bias=None, initial_state=None, cu_seqlens=None, *, dt_softplus: bool = False,
                   return_state: bool = False, out: Optional[Tensor] = None, workspace: Optional[Tensor] = None) -> MambaScanOutputs:
    """Selective scan. For channel d of group g = d // (D / G) and state n, with dt' = dt + dt_bias (through
    softplus with ``dt_softplus``):

        h[t] = exp(dt'[t] a[d, n]) h[t-1] + dt'[t] u[t] b[t, g, n]
        out[t] = (sum_n c[t, g, n] h[t] + d[d] u[t]) * silu(z[t])

    from ``initial_state`` (zeros without it); the skip, gate and bias are left out where d, z, dt_bias are None.

    u, dt, z, out [B, S, D] or packed [T, D]; b, c [..., G, N]; a [D, N], d, dt_bias [D] float32; initial_state
    and the returned ``state`` (with ``return_state``; the last h) [n, D, N] float32, as ``mamba_scan_step``
    takes them. N at most 128. Tokens behind the last sequence: rows of ``out`` are left as they were when
    the caller gives it, else zero."""
    dev = _device("mamba_scan_fwd", "u", u)
    code = _data_dtype("u", u)
    n, S, lead = _sequences("u", u, cu_seqlens, 1)
    D, G, N, (u, dt, b, c, z), (a, d, dt_bias) = _check_scan(u, dt, a, b, c, d, z, dt_bias, lead, dev)
    cu, initial_state = _cu(cu_seqlens, dev), _param("initial_state", initial_state, (n, D, N), _F32, dev)
    res = _out(out, u, u=u, dt=dt, a=a, b=b, c=c, d=d, z=z, dt_bias=dt_bias, initial_state=initial_state, cu_seqlens=cu)
    if workspace is not None:
        _apart("workspace", workspace, u=u, dt=dt, a=a, b=b, c=c, d=d, z=z, dt_bias=dt_bias, initial_state=initial_state, cu_seqlens=cu, out=out)
    state = a.new_empty((n, D, N)) if return_state else None
    packed = cu is not None
    _call("mamba_scan_fwd", (n, S, D, G, N, code, int(bool(dt_softplus)), int(out is None), 0, _ptr(cu), *_rows(u, packed), *_rows(dt, packed),
                             *_rows(b, packed), *_rows(c, packed), *_rows(z, packed), _ptr(a), _ptr(d), _ptr(dt_bias), _ptr(initial_state),
                             _ptr(res), _ptr(state)), dev, workspace)
    return MambaScanOutputs(res, state)


def mamba_scan_bwd(dout, u, dt, a, b, c, d=None, z=None, dt_bias=None, initial_state=None, dstate=None, cu_seqlens=None, *,
                   dt_softplus: bool = False, workspace: Optional[Tensor] = None) -> MambaScanGrads:
    """Gradients of ``sum(out * dout) + sum(state * dstate)`` for the arguments of ``mamba_scan_fwd``: du, ddt,
    db, dc, dz in the data dtype, da, dd, ddt_bias, dinitial_state float32; those of absent inputs are None.
    dout like u, dstate like initial_state. The states are recomputed, so nothing is kept from the forward
    call. Token gradients are zero behind the last sequence."""
    dev = _device("mamba_scan_bwd", "u", u)
    code = _data_dtype("u", u)
    n, S, lead = _sequences("u", u, cu_seqlens, 1)
    D, G, N, (u, dt, b, c, z), (a, d, dt_bias) = _check_scan(u, dt, a, b, c, d, z, dt_bias, lead, dev)
    if dout is None:
        _required(dout=dout)
    dout = _data("dout", dout, u.shape, u.dtype, dev)
    initial_state = _param("initial_state", initial_state, (n, D, N), _F32, dev)
    cu, dstate = _cu(cu_seqlens, dev), _param("dstate", dstate, (n, D, N), _F32, dev)
    if workspace is not None:
        _apart("workspace", workspace, dout=dout, u=u, dt=dt, a=a, b=b, c=c, d=d, z=z, dt_bias=dt_bias, initial_state=initial_state,
               dstate=dstate, cu_seqlens=cu)
    packed = cu is not None
    g = MambaScanGrads(*(None if t is None else _new_like(t) for t in (u, dt, a, b, c, d, z, dt_bias, initial_state)))
    _call("mamba_scan_bwd", (n, S, D, G, N, code, int(bool(dt_softplus)), 0, 0, _ptr(cu), *_rows(dout, packed), *_rows(u, packed),
                             *_rows(dt, packed), *_rows(b, packed), *_rows(c, packed), *_rows(z, packed), _ptr(a), _ptr(d), _ptr(dt_bias),
                             _ptr(initial_state), _ptr(dstate), _ptr(g.du), _ptr(g.ddt), _ptr(g.db), _ptr(g.dc), _ptr(g.dz), _ptr(g.da),
                             _ptr(g.dd), _ptr(g.ddt_bias), _ptr(g.dinitial_state)), dev, workspace)
    return g


def mamba_scan_step(u, dt, state, a, b, c, d=None, z=None, dt_bias=None, state_indices=None, *, dt_softplus: bool = False,
                    out: Optional[Tensor] = None) -> Tensor:
    """One token of ``mamba_scan_fwd`` for each of n rows: u, dt, z, out [n, D]; b, c [n, G, N]; ``state`` [slots,
    D, N] float32 is updated in place. Slots and ``state_indices`` as for ``mamba_conv_step``."""
    dev = _device("mamba_scan_step", "u", u)
    code = _data_dtype("u", u)
    shape = u.shape
    if len(shape) != 2 or 0 in shape:
        raise ValueError(f"u must have shape [n, D] and not be empty, got {list(shape)}")
    n = shape[0]
    D, G, N, (u, dt, b, c, z), (a, d, dt_bias) = _check_scan(u, dt, a, b, c, d, z, dt_bias, (n,), dev)
    slots, stride, idx = _check_pool(state, (D, N), _F32, state_indices, n, dev)
    _apart("state", state, u=u, dt=dt, b=b, c=c, z=z, a=a, d=d, dt_bias=dt_bias, state_indices=idx)
    res = _out(out, u, u=u, dt=dt, a=a, b=b, c=c, d=d, z=z, dt_bias=dt_bias, state=state, state_indices=idx)
    _call("mamba_scan_step", (n, D, G, N, slots, stride, code, int(bool(dt_softplus)), u.data_ptr(), u.stride(0), 0,
                              dt.data_ptr(), dt.stride(0), 0, b.data_ptr(), b.stride(0), 0, c.data_ptr(), c.stride(0), 0,
                              *(_NO_ROWS if z is None else (z.data_ptr(), z.stride(0), 0)),
                              a.data_ptr(), _ptr(d), _ptr(dt_bias), state.data_ptr(), _ptr(idx), res.data_ptr()), dev)
    return res


# ---------------------------------------------------------------- gated group norm
def _row_view(x, D):
    """x [..., D] as rows with one stride: a view where the leading axes allow it, else a copy."""
    x = _dense_inner(x, 1)
    return x.reshape(-1, D) if x.dim() != 2 else x


def _check_norm(what, x, weight, bias, z, groups, eps, gate, activation):
    dev = _device(what, "x", x)
    code = _data_dtype("x", x)
    silu = _activation(activation)
    if gate not in ("before", "after"):
        raise ValueError("gate must be 'before' or 'after'")
    if silu and z is not None:
        raise ValueError("activation and a gate z exclude each other")
    if weight is None:
        _required(weight=weight)
    if x.dim() < 1 or x.numel() == 0:
        raise ValueError(f"x must have shape [..., D] and not be empty, got {list(x.shape)}")
    D = x.shape[-1]
    if isinstance(groups, bool) or not isinstance(groups, int) or groups < 1 or D % groups:
        raise ValueError(f"groups must be a positive int that divides the {D} channels, got {groups!r}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    if D // groups > 8192:
        raise NotImplementedError(f"mamba_norm supports at most 8192 channels in a group, got {D // groups}")
    if z is not None:
        _fits("z", z, x.shape, x.dtype, dev)
        z = _row_view(z, D)
    return dev, code, silu, D, _row_view(x, D), z, _param("weight", weight, (D,), _F32, dev), _param("bias", bias, (D,), _F32, dev)


def mamba_norm_fwd(x, weight, bias=None, z=None, *, groups: int = 1, eps: float = 1e-5, center: bool = False, gate: str = "before",
                   activation: Optional[str] = None, out: Optional[Tensor] = None) -> Tensor:
    """Gated group norm over the last axis, in ``groups`` groups of neighbouring channels (at most 8192 each). With
    v = x * silu(z) (z given, gate "before") or x, and m = mean(v) over the group with ``center``, else 0:

        p = (v - m) / sqrt(mean((v - m)^2) + eps) * weight + bias

    and out = p * silu(z) (z given, gate "after"), silu(p) (activation "silu", without z), or p. x, z, out
    [..., D]; weight, bias [D] float32."""
    dev, code, silu, D, rows, zr, weight, bias = _check_norm("mamba_norm_fwd", x, weight, bias, z, groups, eps, gate, activation)
    res = _out(out, x, x=rows, z=zr, weight=weight, bias=bias)
    _call("mamba_norm_fwd", (rows.shape[0], D, groups, rows.stride(0), 0 if zr is None else zr.stride(0), code, int(bool(center)),
                             int(gate == "after"), silu, eps, 0, _ptr(rows), _ptr(zr), _ptr(weight), _ptr(bias), _ptr(res)), dev)
    return res


def mamba_norm_bwd(dout, x, weight, bias=None, z=None, *, groups: int = 1, eps: float = 1e-5, center: bool = False,
                   gate: str = "before", activation: Optional[str] = None, workspace: Optional[Tensor] = None) -> MambaNormGrads:
    """Gradients of ``sum(out * dout)`` for the arguments of ``mamba_norm_fwd``: dx and dz in x's dtype, dweight and
    dbias float32; dbias and dz are None without the input. The statistics are recomputed from x and z."""
    dev, code, silu, D, rows, zr, weight, bias = _check_norm("mamba_norm_bwd", x, weight, bias, z, groups, eps, gate, activation)
    if dout is None:
        _required(dout=dout)
    _fits("dout", dout, x.shape, x.dtype, dev)
    dr = _row_view(dout, D)
    if workspace is not None:
        _apart("workspace", workspace, dout=dr, x=rows, z=zr, weight=weight, bias=bias)
    dx, dweight = _new_like(x), torch.empty_like(weight)
    dz, dbias = None if z is None else _new_like(z), None if bias is None else torch.empty_like(bias)
    _call("mamba_norm_bwd", (rows.shape[0], D, groups, dr.stride(0), rows.stride(0), 0 if zr is None else zr.stride(0), code,
                             int(bool(center)), int(gate == "after"), silu, eps, 0, _ptr(dr), _ptr(rows), _ptr(zr), _ptr(weight),
                             _ptr(bias), _ptr(dx), _ptr(dz), _ptr(dweight), _ptr(dbias)), dev, workspace)
    return MambaNormGrads(dx, dweight, dbias, dz)
