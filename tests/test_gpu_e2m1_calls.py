"""Calls over an E2M1 cache in the combinations that a serving step makes: the folded
write under a window and without a causal limit, several tokens on a long context, and
a prompt's chunk among requests of several tokens.  The bounds are Batch.check's."""

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from oracle import e2m1
from tests.test_gpu_e2m1 import DEV, Batch, bf16

pytestmark = pytest.mark.gpu


def step(b, splits, seed):
    """Write and attend in one call: against the oracle, the separate calls (the same
    bits), and itself again (the same bits)."""
    rng = np.random.default_rng(seed)
    t = b.dev()
    new = np.concatenate([b.slot_range(r, L - n, L) for r, (L, n) in enumerate(b.lens)])
    kx, vx = (bf16(rng.standard_normal((len(new), b.hkv, b.d))) for _ in range(2))
    kd, vd, slots = kx.to(DEV), vx.to(DEV), torch.from_numpy(new).to(DEV)
    runs = []
    for _ in range(2):
        out, lse = torch.empty_like(t["q"]), torch.empty(t["q"].shape[:2], device=DEV)
        flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkv.pkv_write_attention_varlen_e2m1(kd, vd, slots, t["q"], t["k"], t["v"], out, t["qsl"],
                                            t["lens"], t["table"], b.mq, b.ms, b.scale, b.ks, b.vs,
                                            causal=b.causal, num_splits=splits, lse_out=lse,
                                            error_flag=flag, window=b.window)
        assert flag.item() == 0
        runs.append((out, lse))
    b.k = e2m1.write(b.k, kx.float().numpy(), new, b.ks)
    b.v = e2m1.write(b.v, vx.float().numpy(), new, b.vs)
    assert np.array_equal(t["k"].cpu().numpy(), b.k) and np.array_equal(t["v"].cpu().numpy(), b.v)
    runs.append(b.attend(splits=splits)[:2])
    for out, lse in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    b.check(*runs[0])


TAILS = [(1, 1), (3, 3), (40, 2), (64, 4), (257, 4), (700, 3), (513, 1), (33, 2)]


@pytest.mark.parametrize("splits", [0, 1, 3, 7])
@pytest.mark.parametrize("hq, hkv, d", [(8, 2, 128), (32, 2, 64), (3, 3, 128)])
@pytest.mark.parametrize("window, causal", [(1, True), (3, True), (20, True), (100, True), (300, True),
                                            (20, False), (150, False), (0, False)])
def test_the_folded_write_under_a_window(window, causal, hq, hkv, d, splits):
    step(Batch(TAILS, hq, hkv, d, seed=60, window=window, causal=causal), splits, 61)


@pytest.mark.parametrize("window, causal", [(64, True), (200, True), (0, False), (64, False)])
@pytest.mark.parametrize("d", [64, 128])
def test_a_write_ahead_of_long_requests_under_a_window(window, causal, d):
    step(Batch(TAILS + [(400, 90)], 4, 2, d, seed=62, window=window, causal=causal), 0, 63)


@pytest.mark.parametrize("hq, hkv, d", [(4, 2, 128), (3, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("n", [5, 32, 130])
@pytest.mark.parametrize("window", [0, 100, 3000])
def test_several_tokens_on_a_long_context(n, hq, hkv, d, window):
    b = Batch([(9000, n), (4099, 2), (2500, 17)], hq, hkv, d, seed=64, window=window)
    out, lse, flag = b.attend()
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("window, splits", [(0, 0), (700, 3)])
def test_a_chunk_among_requests_of_several_tokens(window, splits):
    rng = np.random.default_rng(65)
    lens = [(int(rng.integers(300, 1500)), int(rng.integers(2, 5))) for _ in range(31)]
    step(Batch(lens[:15] + [(1300, 400)] + lens[15:], 16, 4, 128, seed=66, window=window), splits, 67)


@pytest.mark.parametrize("hq, hkv", [(128, 1), (64, 2)])
def test_many_query_heads_to_a_kv_head(hq, hkv):
    step(Batch([(300, 4), (77, 3), (1000, 1)], hq, hkv, 128, seed=68), 0, 69)
