"""Long requests over code caches whose score scale leaves fp32's range: a zero or
tiny query row under a small k_scale.  Every score is then 0 to fp32, so a row is
the plain average of the V rows that it sees, whichever kernel takes it."""

import math

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from oracle import fp8
from tests.test_gpu_e2m1 import DECODE, LONG, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [DECODE, LONG])
@pytest.mark.parametrize("hq, hkv, d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("ks", [1e-20, 1e-38])
def test_zero_and_tiny_rows_over_e2m1(lens, hq, hkv, d, ks):
    b = Batch(lens, hq, hkv, d, seed=40, ks=ks)
    b.q[0::3] = 0
    b.q[1::3] *= 2.0 ** -90
    out, lse, flag = b.attend()
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("window", [0, 150])
def test_zero_rows_under_a_window_over_e2m1(window):
    b = Batch(LONG, 4, 2, 128, seed=41, ks=1e-25, window=window)
    b.q[:] = 0
    out, lse, flag = b.attend()
    assert flag.item() == 0
    b.check(out, lse)


@pytest.mark.parametrize("n", [1, 3, 5, 70, 200])
def test_zero_rows_over_e4m3(n):
    """p is 1 (exact), so out is off by the accumulation (2^-23 of the partial sum an
    addition, of V and of p) and the rounding to bf16."""
    L, hq, hkv, d, ks, vs = 300, 4, 2, 128, 1e-20, 0.5
    rng = np.random.default_rng(n)
    nb = -(-L // 16) + 2
    k, v = (rng.integers(0, 0x7F, (nb, 16, hkv, d), dtype=np.uint8) for _ in range(2))
    table = rng.permutation(nb)[: -(-L // 16)].astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    q = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
    pkv.pkv_attention_varlen_e4m3(q, dev(k), dev(v), out, dev(np.array([0, n], np.int32)),
                                  dev(np.array([L], np.int32)), dev(table[None]), n, L, 0.1, ks, vs,
                                  lse_out=lse)
    values = vs * fp8.decode(v)[table].reshape(-1, hkv, d)[:L].astype(np.float64)
    got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy()
    for i in range(n):
        seen = L - n + i + 1
        want = values[:seen].mean(0).repeat(hq // hkv, axis=0)
        assert (np.abs(got[i] - want) <= 2.0 ** -8 * np.abs(want)
                + 2 * L * 2.0 ** -23 * np.abs(values).max()).all()
        assert np.abs(got_lse[i] - math.log(seen)).max() <= 2.0 ** -20 * math.log(seen)
