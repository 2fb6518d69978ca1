"""What the layer operators write must not lie over what they read, index tensors and workspaces among them (no GPU
needed: CPU tensors stand in for device ones)."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from .test_layer_boundary import _conv, _scan, on_cpu  # noqa: F401

Z = torch.zeros
I32, U8 = torch.int32, torch.uint8


def test_output_over_the_index_tensor(on_cpu):  # noqa: F811
    buf = Z(96)
    with pytest.raises(ValueError, match="overlap cu_seqlens"):
        m.mamba_conv_fwd(Z(12, 8), Z(8, 4), out=buf.view(12, 8), cu_seqlens=buf.view(I32)[8:11])
    with pytest.raises(ValueError, match="overlap cu_seqlens"):
        m.mamba_scan_fwd(Z(12, 8), Z(12, 8), Z(8, 4), Z(12, 2, 4), Z(12, 2, 4), out=buf.view(12, 8), cu_seqlens=buf.view(I32)[:3])
    buf = Z(16)
    with pytest.raises(ValueError, match="overlap state_indices"):
        m.mamba_conv_step(Z(2, 8), Z(4, 3, 8), Z(8, 4), state_indices=buf.view(I32)[4:6], out=buf.view(2, 8))
    with pytest.raises(ValueError, match="overlap state_indices"):
        m.mamba_scan_step(Z(2, 8), Z(2, 8), Z(4, 8, 4), Z(8, 4), Z(2, 2, 4), Z(2, 2, 4), state_indices=buf.view(I32)[:2], out=buf.view(2, 8))


def _over(x):
    return x.view(U8).view(-1)


@pytest.mark.parametrize("name", ["dout", "x", "weight", "bias", "initial_state", "dstate"])
def test_workspace_of_the_convolution(on_cpu, name):  # noqa: F811
    a = _conv(dout=Z(2, 6, 8), dstate=Z(2, 3, 8))
    with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
        m.mamba_conv_bwd(**a, workspace=_over(a[name]))


@pytest.mark.parametrize("name", ["u", "dt", "a", "b", "c", "d", "z", "dt_bias", "initial_state", "out", "dout", "dstate"])
def test_workspace_of_the_scan(on_cpu, name):  # noqa: F811
    a = _scan(**({name: Z(2, 6, 8)} if name in ("out", "dout") else {"dout": Z(2, 6, 8), "dstate": Z(2, 8, 4)} if name == "dstate" else {}))
    fn = m.mamba_scan_bwd if "dout" in a else m.mamba_scan_fwd
    with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
        fn(**a, workspace=_over(a[name]))


@pytest.mark.parametrize("name", ["dout", "x", "weight", "bias", "z"])
def test_workspace_of_the_norm(on_cpu, name):  # noqa: F811
    a = dict(dout=Z(3, 8), x=Z(3, 8), weight=Z(8), bias=Z(8), z=Z(3, 8))
    with pytest.raises(ValueError, match=f"workspace must not overlap {name}"):
        m.mamba_norm_bwd(**a, workspace=_over(a[name]))


def test_a_workspace_of_its_own_passes(on_cpu):  # noqa: F811
    with pytest.raises(AssertionError, match="was queued"):
        m.mamba_scan_bwd(**_scan(dout=Z(2, 6, 8)), workspace=Z(64, dtype=U8))
