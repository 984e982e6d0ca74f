"""Row calls of more scale blocks than 32 bits count, and attention captured without a
workspace of its own."""

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from oracle import e2m1
from tests.test_gpu_e2m1 import DEV, Batch

pytestmark = pytest.mark.gpu


def test_more_units_than_32_bits_count():
    """2^28 + 5 rows of one head of 64 in bf16: 2^31 + 40 scale blocks to write, as many
    16-byte pieces to read.  All but six rows are padding."""
    n, d, nb = (1 << 28) + 5, 64, 4
    need = n * (2 * d * 2 + 8) + (8 << 30)
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need >> 30} GB of free device memory")
    rows = [0, 1, (1 << 27) + 3, (1 << 28) - 1, 1 << 28, n - 1]
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((len(rows), 1, d)).astype(np.float32)).bfloat16()
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    at = torch.tensor(rows, device=DEV)
    slots[at] = torch.arange(len(rows), device=DEV) * 7 + 3
    k, v = (torch.empty(n, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[at], v[at] = x.to(DEV), -x.to(DEV)
    caches = [torch.zeros(nb, 1, 9 * d, dtype=torch.uint8, device=DEV) for _ in range(2)]
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.pkv_write_e2m1(k, v, slots, *caches, 0.5, 0.25, error_flag=flag)
    want = np.zeros((nb, 1, 9 * d), dtype=np.uint8)
    for c, y, t in zip(caches, (x, -x), (0.5, 0.25)):
        assert np.array_equal(c.cpu().numpy(), e2m1.write(want, y.float().numpy(), slots[at].cpu().numpy(), t))
    for y in (k, v):
        y[at] = 0
        y[5] = 9.0
    pkv.pkv_read_e2m1(*caches, slots, k, v, 0.5, 0.25, error_flag=flag)
    for c, y, t in zip(caches, (k, v), (0.5, 0.25)):
        got = e2m1.rows(c.cpu().numpy(), slots[at].cpu().numpy(), d, t)
        assert torch.equal(y[at].cpu(), torch.from_numpy(got).float().bfloat16())
        assert (y[5] == 9.0).all()
    assert flag.item() == 0


@pytest.mark.parametrize("lens", [[(3000, 1), (1200, 2)], [(3000, 1), (700, 150)]])
def test_captured_without_a_workspace(lens):
    """The scratch of a captured call belongs to its graph: replays are undisturbed by
    calls and allocations beside them."""
    b = Batch(lens, 8, 2, 128, seed=70)
    t = b.dev()
    want, want_lse, _ = b.attend(t, splits=7)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.attend(t, splits=7, out=out, lse=lse, flag=flag)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        torch.cuda.synchronize()
        g.replay()
        noise = [torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(8)]
        other, other_lse, _ = b.attend(t, splits=7)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert torch.equal(other, want) and torch.equal(other_lse, want_lse)
        assert all((x == 0xFF).all() for x in noise)
    assert flag.item() == 0
