"""Rows over an E2M1 cache that see a NaN key: a NaN output and a NaN log-sum-exp,
whatever the split count and whichever split holds the key.  A NaN value leaves the
log-sum-exp alone."""

import numpy as np
import pytest
import torch

from tests.test_gpu_e2m1 import Batch

pytestmark = pytest.mark.gpu


def scale_byte(b, pos, block):
    slot = int(b.slot_range(0, pos, pos + 1)[0])
    return slot // 16, 8 * b.d + (slot % 16) * (b.d // 16) + block


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 33, 64])
@pytest.mark.parametrize("n", [1, 3])
def test_nan_queries(splits, n):
    b = Batch([(1500, n), (1500, 1)], 4, 2, 128, seed=50)
    b.q[:n, 1] = float("nan")
    out, lse, _ = b.attend(splits=splits)
    want = np.zeros((n + 1, 4), bool)
    want[:n, 1] = True
    assert np.array_equal(lse.isnan().cpu().numpy(), want)
    assert np.array_equal(out.isnan().all(-1).cpu().numpy(), want)
    assert np.array_equal(out.isnan().any(-1).cpu().numpy(), want)
    assert lse[~torch.from_numpy(want).cuda()].isfinite().all()


@pytest.mark.parametrize("splits", [1, 2, 5, 33])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("pos", [0, 700, 1458, 1499])
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_key_in_one_split(splits, n, pos, d):
    b = Batch([(1500, n)], 4, 2, d, seed=51)
    block, at = scale_byte(b, pos, 1)
    b.k[block, 1, at] = 0x7F
    out, lse, _ = b.attend(splits=splits)
    want = np.zeros((n, 4), bool)
    want[np.arange(n) + 1500 - n >= pos, 2:] = True
    assert np.array_equal(lse.isnan().cpu().numpy(), want)
    assert np.array_equal(out.isnan().all(-1).cpu().numpy(), want)
    assert np.array_equal(out.isnan().any(-1).cpu().numpy(), want)


@pytest.mark.parametrize("splits", [1, 4])
@pytest.mark.parametrize("n", [2, 40])
def test_a_nan_value_leaves_the_log_sum_exp(splits, n):
    b = Batch([(1500, n)], 4, 2, 128, seed=52)
    _, clean, _ = b.attend(splits=splits)
    block, at = scale_byte(b, 900, 1)
    b.v[block, 0, at] = 0x7F
    out, lse, _ = b.attend(splits=splits)
    assert torch.equal(lse, clean)
    assert out[:, :2, 16:32].isnan().all() and not out[:, :2, 32:].isnan().any()


def test_a_request_without_a_key_keeps_its_neighbours():
    b = Batch([(40, 1), (0, 0), (33, 2)], 4, 2, 128, seed=53)
    for splits in (1, 3):
        out, lse, flag = b.attend(splits=splits)
        assert flag.item() == 0
        b.check(out, lse)
