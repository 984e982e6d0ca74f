"""Refusals of the E2M1 entry points, on the host: none of these calls reaches
a kernel (every one returns before a launch)."""

import ctypes

import pytest
import torch

import paged_kv_attention_17_gb300 as pkv

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
P = 4096                                                  # an aligned address that is never read


def rows(name, **over):
    a = dict(k_rows=P, v_rows=P, slots=P, n=4, k_cache=P, v_cache=P, blocks=8, bs=16, hkv=2, d=128,
             dtype=1, ks=0.5, vs=0.5, flag=None)
    a.update(over)
    pair, cache = (a["k_rows"], a["v_rows"]), (a["k_cache"], a["v_cache"])
    first, last = (pair, cache) if name == "pkv_write_e2m1" else (cache, pair)
    return getattr(pkv.lib(), name)(*first, a["slots"], a["n"], *last, a["blocks"], a["bs"], a["hkv"],
                                    a["d"], a["dtype"], a["ks"], a["vs"], a["flag"], None)


@pytest.mark.parametrize("name", ["pkv_write_e2m1", "pkv_read_e2m1"])
@pytest.mark.parametrize("over, status", [
    (dict(n=-1), INVALID), (dict(blocks=0), INVALID), (dict(hkv=0), INVALID), (dict(d=0), INVALID),
    (dict(dtype=2), INVALID), (dict(ks=0.0), INVALID), (dict(vs=float("inf")), INVALID),
    (dict(ks=float("nan")), INVALID), (dict(vs=-1.0), INVALID), (dict(bs=32), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(d=16), UNSUPPORTED), (dict(k_rows=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(slots=None), INVALID), (dict(v_rows=P + 8), INVALID),
    (dict(k_cache=P + 4), INVALID), (dict(slots=P + 4), INVALID), (dict(flag=P + 2), INVALID),
    (dict(n=0), 0), (dict(n=0, k_rows=None), 0)])
def test_row_calls(name, over, status):
    assert rows(name, **over) == status


def attend(write=False, **over):
    a = dict(q=P, k=P, v=P, out=P, lse=None, qsl=P, lens=P, table=P, width=4, seqs=2, tokens=2, mq=1,
             ms=64, hq=8, hkv=2, d=128, bs=16, scale=0.1, ks=0.5, vs=0.5, causal=1, window=0,
             splits=1, ws=None, ws_bytes=0, flag=None, blocks=8, k_new=P, v_new=P, slots=P)
    a.update(over)
    tail = [a[x] for x in ("k", "v", "out", "lse", "qsl", "lens", "table", "width", "seqs", "tokens",
                           "mq", "ms", "hq", "hkv", "d", "bs", "scale", "ks", "vs", "causal",
                           "window", "splits", "ws", "ws_bytes", "flag", "blocks")] + [None]
    if write:
        return pkv.lib().pkv_write_attention_varlen_e2m1(a["k_new"], a["v_new"], a["slots"], a["q"], *tail)
    return pkv.lib().pkv_attention_varlen_e2m1(a["q"], *tail)


@pytest.mark.parametrize("write", [False, True])
@pytest.mark.parametrize("over, status", [
    (dict(ks=0.0), INVALID), (dict(vs=float("nan")), INVALID), (dict(window=-1), INVALID),
    (dict(splits=65), INVALID), (dict(splits=-1), INVALID), (dict(hq=7), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(mq=0), INVALID), (dict(width=0), INVALID), (dict(ms=65), INVALID), (dict(q=None), INVALID),
    (dict(table=None), INVALID), (dict(out=P + 2), INVALID), (dict(k=P + 8), INVALID),
    (dict(seqs=65536, tokens=65536), UNSUPPORTED), (dict(blocks=1 << 27), UNSUPPORTED),
    (dict(splits=2), WORKSPACE), (dict(splits=2, ws=P, ws_bytes=100), WORKSPACE),
    (dict(splits=2, ws=P + 16, ws_bytes=1 << 30), WORKSPACE),
    (dict(hq=65536, hkv=65536), UNSUPPORTED),
    (dict(window=64, mq=600000, tokens=600000, width=50000, ms=700000, hq=1, hkv=1), UNSUPPORTED),
    (dict(seqs=0), 0), (dict(tokens=0), 0)])
def test_attention_calls(write, over, status):
    assert attend(write, **over) == status


@pytest.mark.parametrize("over", [dict(k_new=None), dict(slots=None), dict(v_new=P + 8),
                                  dict(slots=P + 4)])
def test_write_and_attend_checks_the_new_rows(over):
    assert attend(True, **over) == INVALID


def test_split_count_rejects_what_it_cannot_size():
    # no device here, or a bad shape: 0, as pkv_num_splits
    assert pkv.lib().pkv_num_splits_e2m1(0, 1, 100, 8, 2, 128, 0) == 0
    assert pkv.lib().pkv_num_splits_e2m1(1, 1, 100, 7, 2, 128, 0) == 0
    assert pkv.lib().pkv_num_splits_e2m1(1, 1, 100, 8, 2, 128, 64) == 0


def test_bindings_refuse_what_is_not_on_the_device():
    cache = torch.zeros(4, 2, 9 * 64, dtype=torch.uint8)
    x = torch.zeros(3, 2, 64)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        pkv.pkv_write_e2m1(x, x, slots, cache, cache, 1.0, 1.0)
    with pytest.raises(ValueError):
        pkv.pkv_read_e2m1(cache, cache, slots, x, x, 1.0, 1.0)


def test_exports_resolve():
    for name in pkv.EXPORTS:
        assert isinstance(getattr(pkv.lib(), name), ctypes._CFuncPtr)
