"""Host model of the E2M1 kernels' index arithmetic: which lane holds which key
and element, that both contractions pair the same ones, that every byte is copied
and every chunk written once, shared-memory bank conflicts, and the order of the
fused write."""

import itertools

import pytest

LANES = range(32)


def kappa(i):
    """Key of MMA row i < 8 of a block (row i + 8: + 8)."""
    return ((i >> 1) ^ 1) + 4 if i & 1 else i >> 1


def v_keys(t4):
    return [t4, (t4 ^ 1) + 4, t4 + 8, (t4 ^ 1) + 12]


def test_keys_of_both_contractions_agree():
    assert sorted(kappa(i) for i in range(8)) == list(range(8))
    for t4 in range(4):
        # the transposed score fragment holds keys kappa(2 t), kappa(2 t + 1), and + 8
        want = [kappa(2 * t4), kappa(2 * t4 + 1), kappa(2 * t4) + 8, kappa(2 * t4 + 1) + 8]
        assert v_keys(t4) == want
    assert sorted(itertools.chain(*(v_keys(t) for t in range(4)))) == list(range(16))


@pytest.mark.parametrize("d", [64, 128])
def test_every_element_enters_the_score_once_on_both_sides(d):
    seen = []
    for t4 in range(4):
        for word in range(d // 32):
            for half in range(2):                        # MMA 2 word + half
                mma = 2 * word + half
                # bytes 2 half, 2 half + 1 of the word: operands a0 / a2
                for operand, byte in enumerate((2 * half, 2 * half + 1)):
                    k_dims = [t4 * (d // 4) + 8 * word + 2 * byte + e for e in range(2)]
                    q_dims = [t4 * (d // 4) + 4 * mma + 2 * operand + e for e in range(2)]
                    assert k_dims == q_dims
                    seen += k_dims
                    # the scale of the word's block is the one that the lane loads
                    block = k_dims[0] // 16
                    assert block == t4 * (d // 64) + (word >> 1 if d == 128 else 0)
    assert sorted(seen) == list(range(d))


@pytest.mark.parametrize("d", [64, 128])
def test_every_output_element_is_one_accumulator_row(d):
    seen = []
    for g in range(8):
        for word in range(d // 64):
            for i in range(4):
                for odd in range(2):                     # even / odd nibbles: rows g, g + 8
                    dim = g * (d // 8) + 8 * word + 2 * i + odd
                    assert dim == g * (d // 8) + 2 * (4 * word + i) + odd
                    assert dim // 16 == g * d // 128     # its scale block
                    seen.append(dim)
    assert sorted(seen) == list(range(d))


def ways(addresses, size):
    """Worst bank conflict of one phase of a shared-memory access."""
    per = 128 // size
    worst = 1
    for p in range(0, len(addresses), per):
        banks = {}
        for a in addresses[p:p + per]:
            if a is not None:
                for b in range(0, size, 4):
                    banks.setdefault((a + b) // 4 % 32, set()).add((a + b) // 4)
        worst = max([worst] + [len(x) for x in banks.values()])
    return worst


@pytest.mark.parametrize("d", [64, 128])
def test_bank_conflicts_of_the_stage_reads(d):
    k = [kappa(lane >> 2) * (d // 2) + (lane & 3) * (d // 8) for lane in LANES]
    assert ways(k, d // 8) == (1 if d == 128 else 2)
    for c in range(4):
        v = [v_keys(lane & 3)[c] * (d // 2) + (lane >> 2) * (d // 16) for lane in LANES]
        assert ways(v, d // 16) <= 2


def swizzle(row, d):
    return (row >> 1) & 3 if d == 128 else ((row >> 1) & 1) | (row & 4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c", [0, 1])
def test_merge_rows_are_stored_without_conflicts_and_read_back(d, c):
    for i in range(0, d // 16, 2):
        at = []
        for lane in LANES:
            row, g = 2 * (lane & 3) + c, lane >> 2
            at.append(row * d * 4 + ((g * (d // 32) + i // 2) ^ swizzle(row, d)) * 16)
        assert ways(at, 16) == 1
    for row in range(16):
        # chunk holds elements 4 chunk .. + 3: accumulators 2 i, 2 i + 1 of tiles i, i + 1
        place = {(chunk ^ swizzle(row, d)): chunk for chunk in range(d // 4)}
        assert len(place) == d // 4
        for lane in LANES:
            chunk = (lane * (d // 32) // 4) ^ swizzle(row, d)
            assert place[chunk] == lane * (d // 32) // 4


@pytest.mark.parametrize("d", [64, 128])
def test_a_stage_is_copied_once(d):
    codes, scales, pair = 8 * d, d, 2
    bytes_seen = []
    for lane in LANES:
        for j in range(pair):
            for which in range(2):                       # K, V
                for c in range(codes // 512):
                    bytes_seen.append(((which * pair + j) * codes + c * 512 + lane * 16,
                                       (which, j, c * 512 + lane * 16)))
        sc = scales // 16
        if lane < 2 * pair * sc:
            p = lane // sc
            bytes_seen.append((2 * pair * codes + lane * 16, (p // pair, p % pair, codes + lane % sc * 16)))
    at = sorted(x for x, _ in bytes_seen)
    assert at == list(range(0, 2 * pair * 9 * d, 16))
    for to, (which, j, source) in bytes_seen:
        p = which * pair + j
        want = p * codes + source if source < codes else 2 * pair * codes + p * scales + source - codes
        assert to == want


@pytest.mark.parametrize("warps", [6, 8])
@pytest.mark.parametrize("splits", [1, 2, 5])
def test_splits_partition_and_no_pair_is_loaded_before_its_new_rows(warps, splits):
    for length in (1, 5, 16, 17, 31, 33, 100, 640, 999):
        for n in range(1, min(4, length) + 1):
            for window in (0, 1, 20, 200):
                kv_lo = max(0, length - n - window + 1) if window else 0
                lo = kv_lo // 16
                nb = -(-length // 16) - lo
                per = -(-nb // splits)
                blocks, stored = [], set()
                for s in range(splits):
                    beg, end = lo + min(nb, s * per), lo + min(nb, (s + 1) * per)
                    blocks += range(beg, end)
                    new_lo, new_hi = max(length - n, max(kv_lo, beg * 16)), min(length, end * 16)
                    stored |= set(range(new_lo, new_hi))
                    npairs = max(0, (end - beg + 1) // 2)
                    for w in range(warps):
                        npw = (npairs - w - 1) // warps + 1 if npairs > w else 0
                        x = new_lo // 16 - beg - 2 * w
                        early = int(x / (2 * warps)) if new_lo < new_hi else npw
                        for k in range(npw):
                            first = beg + 2 * (w + k * warps)
                            if k < early:                # loaded before the barrier
                                assert (first + 2) * 16 <= new_lo or not new_lo < new_hi
                assert blocks == list(range(lo, lo + nb))
                assert stored == set(range(length - n, length))


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_widening_covers_a_tile_without_conflicts(d):
    blocks, units, step = d // 16, 128 * (d // 16) // 64, 64 // (d // 16)
    chunks = {}
    for i in range(units):
        for order in range(2):
            at = []
            for ct in range(64):
                b, r0 = ct % blocks, ct // blocks
                second, c0, r = b >> 2, 2 * (b & 3), r0 + i * step
                chunk = c0 + second if order == 0 else c0 + 1 - second
                assert r & 7 == r0 & 7
                to = second * 16384 + r * 128 + ((chunk ^ (r0 & 7)) << 4)
                word = (second if order == 0 else 1 - second)
                assert word == chunk - c0
                key = (second, r, chunk)
                assert key not in chunks
                chunks[key] = to
                at.append(to)
            assert ways(at[:32], 16) == 1 and ways(at[32:], 16) == 1
        reads = [(r0 + i * step) // 16 * 9 * d + (r0 + i * step) % 16 * (d // 2) + 8 * b
                 for b, r0 in ((ct % blocks, ct // blocks) for ct in range(32))]
        assert ways(reads, 8) == 1
    assert len(chunks) == 128 * d // 8
    assert len(set(chunks.values())) == len(chunks)


def test_edge_tiles_fit_their_notes():
    for pos0 in range(0, 700, 13):                       # first row's position
        for rows in (1, 100, 128, 200, 256):
            for window in (0, 128, 129, 300, 500):
                first = max(0, pos0 - window + 1) if window else 0
                kv_len = pos0 + rows
                base = first // 128
                ntk = -(-kv_len // 128) - base
                last_lo = pos0 + rows - 1 - window + 1 if window else 0
                places = []
                for kt in range(ntk):
                    key0 = (base + kt) * 128
                    if key0 + 128 > pos0 + 1:
                        assert ntk - 1 - kt < 3
                        places.append(ntk - 1 - kt)
                    elif key0 < last_lo:
                        assert kt < 3
                        places.append(3 + kt)
                assert len(set(places)) == len(places)
