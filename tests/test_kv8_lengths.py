"""Lengths up to the last that a table can hold (csrc/kv8_index.h on the CPU, under
the undefined-behaviour sanitiser): tiles of a sequence and the blocks of a run of them."""
import random

import pytest

from .test_kv8_index import X  # noqa: F401 (the compiled header)


@pytest.mark.parametrize("tile", [16, 32, 64])
def test_tiles_and_blocks_of_every_length(X, tile):  # noqa: F811
    rng = random.Random(tile)
    top = 2 ** 31 - 1
    lens = [0, 1, 15, 16, 17, 31, 32, 33, top, top - 1, *(top - 15 - 16 * i for i in range(6))] + [rng.randrange(top) for _ in range(200)]
    for n in lens:
        nt = X.tile_count(n, tile)
        assert nt == -(-n // tile)
        for last in {nt, nt - 1, nt // 2, 1}:
            if 0 < last <= nt:
                assert X.blocks_before(n, last, tile) == -(-min(n, last * tile) // 16)
