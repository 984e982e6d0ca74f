"""Pins of the oracle's 4-bit E2M1 format: closed forms, ties, brute force."""

import numpy as np
import pytest

from oracle import e2m1, fp8


def test_decode_is_the_formats_definition():
    for code in range(16):
        s, e, m = code >> 3, (code >> 1) & 3, code & 1
        mag = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
        assert e2m1.decode(code) == (-mag if s else mag)


@pytest.mark.parametrize("x, code", [
    (0.25, 0), (np.nextafter(0.25, 1), 1), (0.75, 2), (np.nextafter(0.75, 0), 1), (1.25, 2),
    (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (np.nextafter(5.0, 6), 7), (6.0, 7), (1e9, 7),
    (np.inf, 7), (-0.25, 8), (-2.5, 12), (-np.inf, 15), (-0.0, 8)])
def test_encode_ties_and_saturation(x, code):
    assert e2m1.encode(x) == code


def test_encode_inverts_decode():
    c = np.arange(16)
    assert np.array_equal(e2m1.encode(e2m1.decode(c)), c)


def test_quantize_closed_forms():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :16] = 6.0 * 0.5                                # scale 0.5 exactly, codes 6
    x[0, 16:32] = np.tile(np.array([0.5, -1, 1.5, -2, 3, -4, 6, 0]), 2) * 2 * 0.25
    x[0, 32:48] = 1e30                                   # both saturate
    codes, scales = e2m1.quantize(x, 0.5)
    assert scales[0, 0] == fp8.encode(1.0) and (codes[0, :16] == 7).all()
    assert scales[0, 1] == fp8.encode(1.0)
    assert np.array_equal(codes[0, 16:24], [1, 10, 3, 12, 5, 14, 7, 0])
    assert fp8.decode(scales[0, 2]) == 448 and (codes[0, 32:48] == 7).all()
    assert scales[0, 3] == 0 and (codes[0, 48:] == 0).all()
    assert np.array_equal(e2m1.values(codes, scales, 0.5)[0, :32], x[0, :32].astype(np.float64))


def test_quantize_keeps_a_nan_and_bounds_the_error():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)).astype(np.float32)
    x[3, 20] = np.nan
    codes, scales = e2m1.quantize(x, 0.3)
    back = e2m1.values(codes, scales, 0.3)
    assert np.isnan(back[3, 16:32]).all() and np.isfinite(np.delete(back, 3, 0)).all()
    a = np.abs(x).reshape(50, 8, 16).max(-1, keepdims=True)
    err = np.abs(back - x).reshape(50, 8, 16)
    # codes 4 and 6 are furthest apart: half of 2 steps of amax / 6, and the
    # scale's own rounding (2^-4 of at most 6 scales) where it saturates
    assert (err[np.isfinite(err)] <= (np.broadcast_to(a, err.shape) * (1 / 6 + 1 / 16))[np.isfinite(err)]).all()


def test_write_and_rows_round_trip():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (5, 3, 9 * 64), dtype=np.uint8)
    x = rng.standard_normal((4, 3, 64)).astype(np.float32)
    slots = np.array([17, 79, -1, 80])                   # the last two are skipped
    after = e2m1.write(cache, x, slots, 0.7)
    codes, scales = e2m1.quantize(x, 0.7)
    assert np.array_equal(e2m1.rows(after, slots[:2], 64, 0.7), e2m1.values(codes, scales, 0.7)[:2])
    same = np.ones(80, dtype=bool)
    same[[17, 79]] = False
    keep = np.flatnonzero(same)
    assert np.array_equal(e2m1.rows(after, keep, 64, 1.0), e2m1.rows(cache, keep, 64, 1.0), equal_nan=True)
    assert (after != cache).sum() <= 2 * 3 * (32 + 4)


def test_a_planted_scale_mistake_is_caught():
    x = np.linspace(-3, 3, 64, dtype=np.float32)[None]
    codes, scales = e2m1.quantize(x, 1.0)
    assert not np.array_equal(e2m1.values(codes, np.roll(scales, 1, -1), 1.0),
                              e2m1.values(codes, scales, 1.0))
