"""The write + attend call over an E2M1 cache without its new rows is refused before
anything else is looked at: the library function that it calls takes more arguments
than the attention alone, and must never be called with the shorter list."""

import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from paged_kv_attention_17_gb300 import _binding as B


@pytest.mark.parametrize("bad", [None, np.zeros((2, 2, 128), np.float32), 7])
@pytest.mark.parametrize("which, name", [(0, "k_new"), (1, "v_new"), (2, "slot_mapping")])
def test_new_rows_have_to_be_tensors(monkeypatch, which, name, bad):
    monkeypatch.setattr(B, "_device_and_stream", lambda cache, stream: (0, 0))
    rows = [torch.zeros(2, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 128, dtype=torch.bfloat16),
            torch.zeros(2, dtype=torch.int64)]
    rows[which] = bad
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 9 * 128, dtype=torch.uint8)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match=name):
        pkv.pkv_write_attention_varlen_e2m1(*rows, q, cache, cache, q, i32, i32[:2], i32[:2].view(2, 1), 1,
                                            16, 0.1, 0.5, 0.5, num_splits=1)


def test_all_of_them_missing(monkeypatch):
    monkeypatch.setattr(B, "_device_and_stream", lambda cache, stream: (0, 0))
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 9 * 128, dtype=torch.uint8)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError, match="k_new"):
        pkv.pkv_write_attention_varlen_e2m1(None, None, None, q, cache, cache, q, i32, i32[:2],
                                            i32[:2].view(2, 1), 1, 16, 0.1, 0.5, 0.5, num_splits=1)
