"""The scan's kernels in the built library are those that a call can reach (no GPU needed)."""

import itertools
import re

from mamba_mimo_chunked_amd._lib import LIB_PATH

FWD, AGG, AGG2 = 0, 1, 2
SHAPES = [(4, 1), (4, 2), (8, 1), (4, 4), (4, 8), (8, 8), (8, 16)]


def test_walk_instances():
    """By the names of the code objects' symbols (type, states a lane, waves, what is walked, places left out)."""
    names = re.findall(rb"k_walkILi(\d)ELi(\d+)ELi(\d+)ELi(\d)ELb([01])E", LIB_PATH.read_bytes())
    have = {tuple(map(int, m)) for m in names}
    # one wave of eight states: not in the backward walk; places left out: in the outputs' walk alone
    want = {(t, ns, ks, mode, pad) for t, (ns, ks), mode, pad in itertools.product(range(3), SHAPES, (FWD, AGG, AGG2), (0, 1))
            if not (mode == AGG2 and (ns, ks) == (8, 1)) and (mode == FWD or pad == 0)}
    assert have == want
