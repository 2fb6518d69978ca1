"""Which token strides the gated linear recurrence refuses (no GPU needed)."""

import pytest

from mamba_mimo_chunked_amd import _lib

from .test_layer_limits import _query

FAR = (1 << 26) + 8


@pytest.mark.parametrize("fn", ["mamba_recur_fwd", "mamba_recur_bwd"])
@pytest.mark.parametrize("cu", [None, 1 << 20])
def test_a_single_tokens_stride_is_not_used(fn, cu):
    for stride in (FAR, 1 << 40, -64):
        kw = {k: _lib.MambaRows(1 << 20, 64, stride) for k in ("x", "r", "i", "z")}
        if fn.endswith("bwd"):
            kw["dout"] = kw["x"]
        n = 1 if cu else 2
        assert _query(fn, n=n, S=1, cu_seqlens=cu, **kw) == _query(fn, n=n, S=1, cu_seqlens=cu)
        assert _query(fn, n=n, S=1, cu_seqlens=cu, **kw)[0] == _lib.MIMO_OK
        for name in kw:
            assert _query(fn, n=n, S=2, cu_seqlens=cu, **{name: kw[name]})[0] == _lib.MIMO_ERR_UNSUPPORTED
