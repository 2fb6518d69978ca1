"""The workspace of the backward scan, as the size query states it (no GPU needed): it goes by the tokens and the sequences,
not by the tokens of whole chunks that the sequences might fill."""

import ctypes

import pytest

from mamba_mimo_chunked_amd import _lib

from .test_layer_boundary import _args


def _size(**kw):
    kw = dict(initial_state=None, **kw)
    cls, _ = _lib.LAYER_CALLS["mamba_scan_bwd"]
    need = ctypes.c_size_t(0)
    st = _lib.lib().mamba_scan_bwd_workspace_size(ctypes.byref(_args(cls, **kw)), ctypes.byref(need))
    assert st == _lib.MIMO_OK, _lib.last_error()
    return need.value


def _chunk(n, S, D, G, N, packed):
    """Channels of a tile, and tokens of a chunk: 128, halved while fewer than 1024 blocks would walk, down to 16; a
    whole sequence of up to 128 tokens where two chunks would hold it."""
    tile = 128 if N <= 8 else 64 if N <= 32 else 32 if N <= 64 else 16
    tiles, T, C = -(-(D // G) // tile), S if packed else n * S, 128
    while C > 16 and T // C * G * tiles < 1024:
        C //= 2
    return tiles, T, 128 if S <= min(128, 2 * C) else C


def _stated(n, S, D, G, N, packed):
    """What the header states, in bytes."""
    tiles, T, C = _chunk(n, S, D, G, N, packed)
    chunks = S // C + n + 1 if packed else n * -(-S // C)
    cut = S > C
    units = 0 if S <= 16 or C == 16 else S * (C // 16 - 1) // C + n if packed else n * (-(-S // 16) - -(-S // C))
    return 8 * G * N * tiles * T + 4 * D * chunks * (N + 2 + (N + 1 if cut else 0)) + 4 * D * units * (N + 1)


SHAPES = [  # n, S, D, G, N, packed
    (1, 16000, 2048, 1, 16, True), (2000, 16000, 2048, 1, 16, True), (1024, 20, 4096, 1, 128, False), (4, 4096, 1024, 1, 16, False),
    (3, 903, 200, 2, 24, True), (1, 1, 8, 1, 1, False), (7, 4100, 2048, 4, 64, True), (64, 17, 64, 1, 8, False), (64, 128, 64, 1, 8, False),
    (64, 129, 64, 1, 8, False), (5, 16, 64, 1, 8, False), (1, 100000, 1024, 128, 16, False),
]


@pytest.mark.parametrize("n,S,D,G,N,packed", SHAPES)
def test_workspace_is_what_the_header_states(n, S, D, G, N, packed):
    got = _size(n=n, S=S, D=D, G=G, N=N, cu_seqlens=1 << 20 if packed else None)
    want = _stated(n, S, D, G, N, packed)
    assert want <= got <= want + 7 * 256        # seven parts, each in whole 256 bytes


def test_many_short_sequences():
    """The same tokens in 2000 sequences instead of one: a state for each, not eight."""
    D, N, T = 2048, 16, 16000
    one, many = (_size(n=n, S=T, D=D, G=1, N=N, cu_seqlens=1 << 20) for n in (1, 2000))
    assert many - one <= 2000 * 4 * D * (3 * (N + 1) + 1) + 8 * 256
    # sequences of 20 tokens, one unit behind the first: a state more each, beside the sums
    assert _size(n=1024, S=20, D=4096, G=1, N=128) <= 1024 * 4096 * 4 * (2 * 128 + 4) + 1024 * 20 * 8 * 128 * 256 + 8 * 256
