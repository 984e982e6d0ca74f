"""Calls on streams given by argument that bring no workspace: two streams at once,
neither of them current, held back while the current stream allocates and fills
blocks of the workspace's size.  The results are the bits of a call by itself."""

import pytest
import torch

import paged_kv_attention_17_gb300 as pkv

pytestmark = pytest.mark.gpu

HQ, HKV, D, L, SEQS, SPLITS = 8, 2, 128, 2000, 3, 7
CACHES = ["bf16", "e4m3", "e2m1", "cascade"]


def problem(cache, seed):
    """A function of (stream, out, lse) that makes one call without a workspace, and
    the workspace's size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = -(-L // 16)
    n = SEQS * blocks
    table = torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(SEQS, blocks)
    q = torch.randn(SEQS, HQ, D, generator=g, device="cuda").bfloat16()
    qsl = torch.arange(SEQS + 1, device="cuda", dtype=torch.int32)
    lens = torch.full((SEQS,), L, dtype=torch.int32, device="cuda")
    if cache in ("bf16", "cascade"):
        k, v = (torch.randn(n, 16, HKV, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        call, more = pkv.pkv_attention_varlen, ()
    elif cache == "e4m3":
        k, v = (torch.randint(0, 0x7F, (n, 16, HKV, D), generator=g, device="cuda").to(torch.uint8)
                for _ in range(2))
        call, more = pkv.pkv_attention_varlen_e4m3, (0.01, 0.5)
    else:
        k, v = (torch.randint(0, 0x60, (n, HKV, 9 * D), generator=g, device="cuda").to(torch.uint8)
                for _ in range(2))
        call, more = pkv.pkv_attention_varlen_e2m1, (0.01, 0.5)

    if cache == "cascade":
        suffix, own = lens - 1600, table[:, 100:].contiguous()
        size = pkv.pkv_cascade_workspace_bytes(SEQS, HQ, D, SPLITS)
    else:
        size = pkv.pkv_workspace_bytes(SEQS, HQ, D, SPLITS)

    def run(stream, out, lse):
        if cache == "cascade":
            pkv.pkv_cascade_attention(q, k, v, out, qsl, suffix, own, table[0, :100], 1, L - 1600, 0.1,
                                      prefix_splits=SPLITS, lse_out=lse, stream=stream)
        else:
            call(q, k, v, out, qsl, lens, table, 1, L, 0.1, *more, num_splits=SPLITS, lse_out=lse,
                 stream=stream)

    return run, size


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("cache", CACHES)
def test_two_streams_without_workspaces(cache, raw):
    problems = [problem(cache, seed) for seed in (1, 2)]
    new = lambda: (torch.zeros(SEQS, HQ, D, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                   torch.zeros(SEQS, HQ, device="cuda"))
    want = []
    for run, _ in problems:
        out, lse = new()
        run(None, out, lse)
        want.append((out, lse))
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in problems]
    assert not torch.equal(want[0][0], want[1][0])
    for _ in range(3):
        got = [new() for _ in problems]
        torch.cuda.synchronize()
        for side in sides:                                 # (some 5 ms)
            with torch.cuda.stream(side):
                torch.cuda._sleep(10_000_000)
        noise = []
        for (run, size), side, (out, lse) in zip(problems, sides, got):
            run(side.cuda_stream if raw else side, out, lse)
            noise += [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        for side, (out, lse), (w_out, w_lse) in zip(sides, got, want):
            side.synchronize()
            assert torch.equal(out, w_out) and torch.equal(lse, w_lse)
        assert all((x == 0xFF).all() for x in noise)


def test_the_legacy_stream_by_its_handle():
    run, _ = problem("e2m1", 3)
    outs = []
    for stream in (None, 0, torch.cuda.default_stream()):
        out = torch.zeros(SEQS, HQ, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(SEQS, HQ, device="cuda")
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            run(stream, out, lse)
        torch.cuda.synchronize()
        outs.append((out, lse))
    assert outs[0][0].isfinite().all()
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
