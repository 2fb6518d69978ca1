"""The refusals of the residual addition's norm name the tensor that is at fault (no GPU needed)."""

import pytest
import torch

import mamba_mimo_chunked_amd as m

from .test_layer_boundary import on_cpu  # noqa: F401

Z = torch.zeros


def test_an_empty_tensor_is_named(on_cpu):  # noqa: F811
    for shape in ((0, 8), (3, 0), ()):
        with pytest.raises(ValueError, match="^x must have shape"):
            m.mamba_add_norm_fwd(Z(shape), Z(8))
        with pytest.raises(ValueError, match="^dout must have shape"):
            m.mamba_add_norm_bwd(Z(shape), Z(shape), Z(8))
