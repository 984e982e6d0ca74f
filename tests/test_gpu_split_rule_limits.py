"""The split rules at the ends of their arguments' types: rows whose 32-bit
product would wrap are a full grid."""

import pytest

import paged_kv_attention_17_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq", [(1 << 30) + 1, (1 << 30) + 300, (1 << 31) - 1, 1 << 29])
@pytest.mark.parametrize("rule", [pkv.pkv_num_splits, pkv.pkv_num_splits_e2m1])
def test_a_full_grid_is_not_split(rule, hq):
    for tokens in (1, 2, 4):
        assert rule(1, tokens, 1 << 20, hq, 1, 128) == 1
