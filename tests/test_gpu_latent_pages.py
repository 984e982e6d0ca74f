"""Block tables of absorbed latent attention that name no block of the cache."""

import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from tests.test_gpu_latent import attend, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -2, -3, -(1 << 31), 83, (1 << 31) - 1])
def test_any_entry_outside_the_cache_is_flagged(bad):
    """Whatever the value, wherever in the context it stands; behind a context it is not
    looked at.  (83 blocks.)"""
    c = case([200, 1000, 40], [1, 3, 1], 16, 19, spare=4)
    assert c["cache"].shape[0] == 83
    want, wlse = attend(c)
    for r, at in ((0, 0), (0, 12), (1, 5), (1, 62), (2, 2)):
        table = c["table"].clone()
        table[r, at] = bad
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = attend(c, flag=flag, table=table)
        assert int(flag) == pkv.FLAG_BAD_BLOCK, (r, at)
        keep = torch.ones(5, dtype=torch.bool, device="cuda")
        keep[int(c["qsl"][r]):int(c["qsl"][r + 1])] = False
        assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], wlse[keep])
    table = c["table"].clone()
    table[0, 13:], table[2, 3:] = bad, bad
    got = attend(c, table=table)
    assert torch.equal(got[0], want) and torch.equal(got[1], wlse)
