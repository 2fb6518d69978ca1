"""Sizes that the layer operators cannot take are refused before anything is queued (no GPU needed): the size queries refuse
what the calls refuse, and what needs many threads along one axis only for its last kernel is not refused at all."""

import ctypes

import pytest

from mamba_mimo_chunked_amd import _lib

from .test_layer_boundary import _args


def _query(fn, **kw):
    cls, _ = _lib.LAYER_CALLS[fn]
    need = ctypes.c_size_t(0)
    return getattr(_lib.lib(), fn + "_workspace_size")(ctypes.byref(_args(cls, **kw)), ctypes.byref(need)), need.value


@pytest.mark.parametrize("fn,kw", [
    # 2^29 chunks of 128 tokens, of a wave or more each
    ("mamba_scan_bwd", dict(n=65535, S=1 << 20, D=1, G=1, N=1)), ("mamba_scan_bwd", dict(n=65535, S=1 << 17, D=2, G=1, N=4)),
])
def test_more_than_2_32_threads_are_refused_by_the_query(fn, kw):
    assert _query(fn, **kw)[0] == _lib.MIMO_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(n=256, S=1024, D=64, G=64, N=128), dict(n=1, S=1 << 22, D=512, G=8, N=64)])
def test_many_elements_of_db_and_dc_are_accepted(kw):
    """2^32 of them and more."""
    assert kw["n"] * kw["S"] * kw["G"] * kw["N"] * 2 >= 1 << 32
    st, need = _query("mamba_scan_bwd", **kw)
    assert st == _lib.MIMO_OK and need > 1 << 34
