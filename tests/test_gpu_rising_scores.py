"""Prefill rows whose reference maximum moves at every key tile.

The scores of a row rise (or fall, or both beside each other in one warp) along the
context, so that the accumulator is rescaled again and again while the next tile's
products are being made; over each type of cache, against the formula in 64 bits.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_17_gb300 as pkv
from oracle import e2m1

pytestmark = pytest.mark.gpu

DEV = "cuda"
KS, VS = 0.5, 0.3


def oracle(q, K, V, qsl, lens, scale):
    """(o, X, V's maximum): o per row and head, X the largest sum of |q k| of a row."""
    o, top = np.zeros(q.shape), np.zeros(q.shape[:2])
    group = q.shape[1] // K[0].shape[1]
    for r, L in enumerate(lens):
        a, b = qsl[r], qsl[r + 1]
        see = np.arange(L) <= (L - (b - a) + np.arange(b - a))[:, None]
        for h in range(q.shape[1]):
            k, v = K[r][:, h // group], V[r][:, h // group]
            s = np.where(see, scale * (q[a:b, h] @ k.T), -np.inf)
            w = np.exp(s - s.max(1, keepdims=True))
            o[a:b, h] = (w @ v) / w.sum(1, keepdims=True)
            top[a:b, h] = (scale * (np.abs(q[a:b, h]) @ np.abs(k).T)).max(1)
    return o, top, max(np.abs(v).max() for v in V)


@pytest.mark.parametrize("d, hq, hkv", [(128, 4, 2), (128, 3, 1), (64, 4, 1)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("lens", [[(1500, 700), (131, 131)], [(2049, 40)]])
def test_rising_and_falling_scores(kind, d, hq, hkv, lens):
    rng = np.random.default_rng(3)
    ctx = [L for L, _ in lens]
    qsl = np.concatenate([[0], np.cumsum([n for _, n in lens])]).astype(np.int32)
    counts = [-(-L // 16) for L in ctx]
    nb = sum(counts) + 2
    perm = rng.permutation(nb).astype(np.int32)
    table = np.zeros((len(lens), max(counts)), np.int32)
    at, slots = 0, []
    for r, c in enumerate(counts):
        table[r, :c] = perm[at:at + c]
        at += c
        p = np.arange(ctx[r])
        slots.append(table[r][p // 16].astype(np.int64) * 16 + p % 16)
    flat = np.concatenate(slots)

    scale = 1.0 / np.sqrt(d)
    u = rng.choice([-1.0, 1.0], (hkv, d))
    step = 0.1 / (scale * d)                               # a score moves by 0.1 a key
    k = np.concatenate([u * (step * np.arange(L))[:, None, None] for L in ctx])
    v = rng.standard_normal(k.shape)
    c = np.array([1.0, -1.0, 0.5, 2.0])[rng.integers(0, 4, (qsl[-1], hq))]
    q = torch.from_numpy(np.repeat(u, hq // hkv, axis=0) * c[..., None]).to(torch.bfloat16)

    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    args = dict(qsl=t(qsl), lens=t(np.array(ctx, np.int32)), table=t(table))
    mq, ms = max(n for _, n in lens), max(ctx)
    qd = q.to(DEV)
    out = torch.empty_like(qd)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    tail = (args["qsl"], args["lens"], args["table"], mq, ms, scale)
    if kind == "e2m1":
        caches = [e2m1.write(np.full((nb, hkv, 9 * d), 0x7F, np.uint8), x.astype(np.float32), flat, s)
                  for x, s in ((k, KS), (v, VS))]
        K, V = ([e2m1.rows(x, sl, d, s) for sl in slots] for x, s in zip(caches, (KS, VS)))
        pkv.pkv_attention_varlen_e2m1(qd, t(caches[0]), t(caches[1]), out, *tail, KS, VS,
                                      error_flag=flag)
    else:
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        caches = []
        for x in (k, v):
            full = torch.full((nb * 16, hkv, d), float("nan")).to(dt)
            full[torch.from_numpy(flat)] = torch.from_numpy(x).float().to(dt)
            caches.append(full.view(nb, 16, hkv, d))
        K, V = ([x.float().view(nb * 16, hkv, d)[torch.from_numpy(sl)].numpy().astype(np.float64)
                 for sl in slots] for x in caches)
        if kind == "bf16":
            pkv.pkv_attention_varlen(qd, caches[0].to(DEV), caches[1].to(DEV), out, *tail,
                                     error_flag=flag)
        else:
            pkv.pkv_attention_varlen_e4m3(qd, caches[0].view(torch.uint8).to(DEV),
                                          caches[1].view(torch.uint8).to(DEV), out, *tail, 1.0, 1.0,
                                          error_flag=flag)
    o, X, top_v = oracle(q.float().numpy().astype(np.float64), K, V, qsl, ctx, scale)
    # the output's rounding, P's (bf16 2^-8, f16 2^-11 and half its least subnormal for
    # each key, against a sum of at least 1), and the scores' 32-bit sums in numerator
    # and denominator
    rel = (d + 8) * 2.0 ** -23 * (X + 8)
    p = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11 + ms * 2.0 ** -25
    tol = 2.0 ** -8 * np.abs(o) + ((2 * p + 2 * rel) * top_v)[..., None]
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - o)
    assert flag.item() == 0
    assert (err <= tol).all(), (err - tol).max()
