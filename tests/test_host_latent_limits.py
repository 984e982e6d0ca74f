"""How many keys an expanded call takes: a tile's end stays within 32 bits.  None of these
calls reaches a kernel."""

import pytest

from tests.test_host_latent import INVALID, UNSUPPORTED, expanded

TILE = 128


def test_the_last_tile_of_as_many_keys_as_are_taken_ends_within_32_bits():
    most = 1 << 30
    assert expanded(keys=most, k=None) == INVALID          # (within the limit: the rows are looked at)
    # a request's tiles begin at its first key, wherever that lies: its last tile's end
    assert max(start + -(-(most - start) // TILE) * TILE for start in (0, 1, most - 1, most // 2 + 5)) < 1 << 31


@pytest.mark.parametrize("keys", [(1 << 30) + 1, (1 << 31) - 1, 1 << 40])
def test_more_keys_are_refused(keys):
    assert expanded(keys=keys, k=None) == UNSUPPORTED
