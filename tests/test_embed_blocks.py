"""Sizes of the token embedding whose launches would have 2^31 blocks or more are refused (no GPU). A block
zeroes 16 KB of the gradient's rows, 32 rows at most and one at least.
"""
import pytest

import context_parallelism_gb300 as up
from tests.test_embed_api import INV, UNS, _bwd, _fwd

MOST = (1 << 31) - 1


@pytest.mark.parametrize("S,Dm,V,fits", [
    (8, 8, MOST, True), (8, 2048, MOST, True),             # 32 rows and 2 rows a block
    (1, 4096, MOST - 4, True), (8, 4096, MOST, False),     # one row, beside the places' chunks
    (1, 8192, MOST, False),
    (1, 1 << 24, MOST - 16384, True),                      # one row, 16384 blocks a chunk
    (1, 1 << 24, MOST - 16383, False), (1, 1 << 24, 1 << 30, True),
])
def test_blocks_of_the_gradient(S, Dm, V, fits):
    assert (up.upipe_embed_workspace_bytes(S, Dm, V) > 0) == fits
    assert _bwd(S=S, Dm=Dm, V=V, wb=1 << 60) == (INV if fits else UNS)  # (no device memory)
    assert _fwd(S=S, Dm=Dm, V=V) == INV
