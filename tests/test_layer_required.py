"""A tensor that a layer operator cannot do without is asked for by name (no GPU needed)."""

import pytest
import torch

from mamba_mimo_chunked_amd import layer

from .test_layer_boundary import PY

NEEDED = {"mamba_conv_fwd": ("x", "weight"), "mamba_conv_bwd": ("dout", "x", "weight"), "mamba_conv_step": ("x", "state", "weight"),
          "mamba_scan_fwd": ("u", "dt", "a", "b", "c"), "mamba_scan_bwd": ("dout", "u", "dt", "a", "b", "c"),
          "mamba_scan_step": ("u", "dt", "state", "a", "b", "c"), "mamba_norm_fwd": ("x", "weight"), "mamba_norm_bwd": ("dout", "x", "weight")}


@pytest.mark.parametrize("fn,make,name", [(f, mk, k) for f, mk, _ in PY for k in NEEDED[f.__name__]])
def test_missing_tensor(monkeypatch, fn, make, name):
    device = layer._device      # the check itself for an absent tensor; CPU tensors stand in for device ones
    monkeypatch.setattr(layer, "_device", lambda what, n, x: device(what, n, x) if x is None else x.device)
    monkeypatch.setattr(layer, "_call", lambda *a: pytest.fail("was queued"))
    assert isinstance(make()[name], torch.Tensor)
    with pytest.raises(ValueError, match=f"{name} is required"):
        fn(**make(**{name: None}))
