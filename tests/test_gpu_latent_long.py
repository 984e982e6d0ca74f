"""Contexts so long that a block's share of one takes longer than a single wait's limit."""

import pytest
import torch

import paged_kv_attention_17_gb300 as pkv

pytestmark = pytest.mark.gpu


def test_pieces_of_more_than_two_seconds():
    """160 contexts of 10^8 keys over the same 64 blocks: 1.5 million tiles each, 2.4 s at 1.5 us,
    and a next one behind them in the first block.  Equal scores; half of the keys hold a one in
    the latent's second half, whose sums (5 10^7) fp32 holds exactly."""
    n, keys, hq = 160, 100_000_000, 16
    table = (torch.arange(keys // 16, device="cuda", dtype=torch.int32) % 64).repeat(n, 1)
    cache = torch.zeros(64, 16, 576, dtype=torch.bfloat16, device="cuda")
    cache[::2, :, 256:512] = 1.0
    out = torch.full((n, hq, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse, flag = torch.zeros(n, hq, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.pkv_latent_attention_varlen(
        torch.zeros(n, hq, 576, dtype=torch.bfloat16, device="cuda"), cache, out,
        torch.arange(n + 1, dtype=torch.int32, device="cuda"),
        torch.full((n,), keys, dtype=torch.int32, device="cuda"), table, 1, keys, 0.07, lse_out=lse, error_flag=flag)
    assert int(flag) == 0
    assert bool((out[..., :256] == 0).all())
    # a merge's weights are off by 2^-18, the row is rounded to bf16 (2^-8 of it)
    assert float((out[..., 256:].double() - 0.5).abs().max()) <= 0.5 * (2.0 ** -8 + 2.0 ** -18)
    want = torch.tensor(float(keys), dtype=torch.float64).log().item()
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -18
