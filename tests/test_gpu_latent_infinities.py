"""Infinities and NaN in keys that a row of absorbed latent attention sees: the result does
not depend on where in a context, a unit or a tile the key lies."""

import numpy as np
import pytest
import torch

from oracle import latent as L
from tests.test_gpu_latent import SCALE, attend, case, check, oracle

pytestmark = pytest.mark.gpu
INF = float("inf")


def slots_of(c, r, j):
    return c["table"][r].long()[j // 16] * 16 + j % 16


def without(c, gone, causal=True, scale=SCALE):
    """The oracle of each request over its keys but those of the list gone[r]."""
    d = lambda x: x.double().cpu().numpy()  # noqa: E731
    q, rows, hq, parts = d(c["q"]), c["cache"].view(-1, 576), c["q"].shape[1], []
    for r, length in enumerate(c["lens"].tolist()):
        a, b = c["qsl"][r:r + 2].tolist()
        j = np.arange(length)
        keys = d(rows[slots_of(c, r, torch.arange(length, device="cuda"))])
        at = length - (b - a) + np.arange(b - a)
        seen = (j <= at[:, None] if causal else np.ones((b - a, length), bool)) & ~np.isin(j, gone[r])
        keys[gone[r]] = 0.0
        parts += [(a, h, L._attend(q[a:b, h], keys, keys[:, :512], scale, seen)) for h in range(hq)]
    return L._rows(parts, q.shape[0], hq, 512)


def sees(c, r, key, causal=True):
    """The rows (tokens) of the batch that see key `key` of request r."""
    a, b = c["qsl"][r:r + 2].tolist()
    at = int(c["lens"][r]) - (b - a) + np.arange(b - a)
    out = np.zeros(c["q"].shape[0], bool)
    out[a:b] = at >= key if causal else True
    return out


def check_but(out, lse, got, nan):
    """`nan`: the elements that are NaN; the others within the bounds."""
    have = np.isnan(out.double().cpu().numpy())
    assert np.array_equal(have, nan), (int(have.sum()), int(nan.sum()))
    keep = torch.from_numpy(~nan).cuda()
    check(torch.where(keep, out, torch.zeros_like(out)), lse, tuple(
        np.where(nan, 0.0, x) if x.ndim == 3 else x for x in got))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens, news, hq, places", [
    ([200], [2], 4, (5, 77, 193, 198, 199)), ([100], [40], 1, (0, 59, 60, 61, 75, 99)),
    ([333, 64], [30, 1], 4, (100, 303, 304, 318, 319, 332)), ([9000], [3], 16, (10, 4500, 8990, 8998, 8999)),
    ([64, 40], [1, 2], 16, (0, 63)), ([700] * 12, [1] * 12, 16, (3, 650, 699))])
def test_a_key_scored_minus_infinity(lens, news, hq, places, causal):
    """A key with an infinity, scored -inf, weighs 0: the elements where its latent part holds
    an infinity are NaN (0 times it) in the rows that see it and only there, wherever the key
    lies; with the infinity in its positional part no element is."""
    c = case(lens, news, hq, 30 + len(places))
    c["q"][..., 100], c["q"][..., 300], c["q"][..., 570] = 1.0, -2.0, 1.0
    rows, clean = c["cache"].view(-1, 576), c["cache"].clone()
    for key in places:
        for holds in ({100: -INF}, {300: INF}, {100: -INF, 300: INF}, {570: -INF}, {570: -INF, 300: INF}):
            c["cache"].copy_(clean)
            for e, x in holds.items():
                rows[slots_of(c, 0, torch.tensor(key)), e] = x
            got = without(c, [[key]] + [[]] * (len(lens) - 1), causal)
            nan = np.zeros((c["q"].shape[0], hq, 512), bool)
            for e in holds:
                if e < 512:
                    nan[sees(c, 0, key, causal), :, e] = True
            check_but(*attend(c, causal), got, nan)


@pytest.mark.parametrize("e, x", [(100, INF), (300, -INF), (570, INF), (200, INF),
                                  (100, float("nan")), (570, float("nan"))])
def test_a_key_scored_plus_infinity_or_nan(e, x):
    """Its row of the output is NaN, the log-sum-exp too (as 0 times an infinity is, element 200);
    rows that do not see the key, in its tile or not, stay as they are."""
    for lens, news, hq, places in (([200], [2], 4, (5, 77, 193, 199)), ([100], [40], 1, (0, 61, 75, 99)),
                                   ([333, 64], [30, 1], 4, (100, 303, 304, 319, 332)), ([9000], [3], 16, (4500, 8999))):
        c = case(lens, news, hq, 40)
        c["q"][..., 100], c["q"][..., 300], c["q"][..., 570], c["q"][..., 200] = 1.0, -2.0, 1.0, 0.0
        clean, want = c["cache"].clone(), oracle(c)
        for key in places:
            c["cache"].copy_(clean)
            c["cache"].view(-1, 576)[slots_of(c, 0, torch.tensor(key)), e] = x
            out, lse = attend(c)
            see = torch.from_numpy(sees(c, 0, key)).cuda()
            assert bool(torch.isnan(out[see]).all()) and bool(torch.isnan(lse[see]).all())
            keep = (~see).cpu().numpy()
            check(out[~see], lse[~see], tuple(w[keep] for w in want))


@pytest.mark.parametrize("length, first, last", [(9000, 0, 4000), (9000, 5000, 9000), (9000, 0, 9000), (50, 0, 50), (50, 0, 49)])
def test_whole_runs_of_keys_scored_minus_infinity(length, first, last):
    """Long enough that some of the context's pieces see no other key.  Without any other
    key at all a row is 0, its log-sum-exp -inf."""
    c = case([length], [2], 8, 41)
    c["q"][..., 570] = 1.0
    rows = c["cache"].view(-1, 576)
    rows[slots_of(c, 0, torch.arange(first, last, device="cuda")), 570] = -INF
    gone = [list(range(first, last))]
    nan = np.zeros((2, 8, 512), bool)
    check_but(*attend(c), without(c, gone), nan)
    for key in (first + 3, last - 20):
        rows[slots_of(c, 0, torch.tensor(key)), 200] = INF
    nan[..., 200] = True
    c["q"][..., 200] = -1.0
    check_but(*attend(c), without(c, gone), nan)
