"""Every key tile's share in latent attention, read off the output, and requests beside one
that is told of as invalid."""

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from tests.test_gpu_latent import attend, case, expand, wide

pytestmark = pytest.mark.gpu


def slots_of(c, r, j):
    return c["table"][r].long()[j // 16] * 16 + j % 16


@pytest.mark.parametrize("lens, news, hq", [
    ([32767], [1], 16), ([32768, 5000], [1, 1], 16), ([32700], [3], 128), ([20001, 77, 31000], [2, 1, 4], 20),
    ([2000] * 64, [1] * 64, 32)])
def test_every_tile_has_its_share(lens, news, hq):
    """Equal scores, and tile t of 64 keys holds ones in element t alone: an element is its
    tile's share of the keys that the row sees.  All terms are exact (p is 1 or, against a
    piece's maximum, 2^0); a merge's weights are off by 2^-19 each (numerator and sum), and the row is
    rounded to bf16 once: 2^-8 of it."""
    c = case(lens, news, hq, 50)
    c["q"].zero_()
    c["cache"].zero_()
    rows = c["cache"].view(-1, 576)
    for r, n in enumerate(lens):
        j = torch.arange(n, device="cuda")
        rows[slots_of(c, r, j), j // 64] = 1.0
    out, lse = attend(c)
    out, t = out.double().cpu().numpy(), 0
    for r, n in enumerate(lens):
        for i in range(news[r]):
            seen = n - news[r] + i + 1
            want = np.clip(seen - 64 * np.arange(512), 0, 64) / seen
            assert np.all(np.abs(out[t] - want) <= (2.0 ** -8 + 2.0 ** -18) * want), (r, i)
            assert np.all(np.abs(lse[t].double().cpu().numpy() - np.log(seen)) <= 2.0 ** -18)
            t += 1


@pytest.mark.parametrize("news, keys, hq", [([1], [16384], 3), ([300, 20], [16000, 129], 2), ([400, 130], [9000, 4001], 80)])
def test_every_tile_of_expanded_keys_has_its_share(news, keys, hq):
    """The same with tiles of 128 keys and values of 128 elements."""
    c = wide(news, keys, hq, 51, dense=True)
    c["q"].zero_()
    c["v"].zero_()
    at = 0
    for m in keys:
        j = torch.arange(m, device="cuda")
        c["v"][at + j, :, j // 128] = 1.0
        at += m
    out, lse = expand(c)
    out, t = out.double().cpu().numpy(), 0
    for r, m in enumerate(keys):
        seen = m - news[r] + 1 + np.arange(news[r])
        want = np.clip(seen[:, None] - 128 * np.arange(128), 0, 128) / seen[:, None]
        got = out[t:t + news[r]]
        assert np.all(np.abs(got - want[:, None]) <= (2.0 ** -8 + 2.0 ** -18) * want[:, None]), r
        t += news[r]


def test_expanded_requests_beside_an_invalid_one():
    """A request that is told of writes none of its neighbours' rows, nor they its."""
    c = wide([10, 20, 7], [30, 40, 9], 2, 52)
    want, wlse = expand(c)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for over, valid in ((dict(ksl=ints(0, 30, 100, 105)), [0]), (dict(mk=35), [0, 2]), (dict(mq=15), [0, 2]),
                        (dict(ksl=ints(0, -1, 70, 79)), [2]), (dict(ksl=ints(0, 30, 70, 3)), [0, 1])):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = expand(c, flag=flag, **over)
        assert int(flag) == pkv.FLAG_BAD_LENGTHS, over
        for r in range(3):
            rows = slice(int(c["qsl"][r]), int(c["qsl"][r + 1]))
            if r in valid:
                assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wlse[rows]), (over, r)
            else:
                assert bool((out[rows] == 7).all()) and bool((lse[rows] == 7).all()), (over, r)
