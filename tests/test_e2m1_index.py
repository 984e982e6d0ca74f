"""The E2M1 kernels' index arithmetic, as csrc/e2m1_index.h has it for the kernels,
compiled for the host: both contractions take the same keys, every byte of a stage is
copied once and every byte of its rows read by one lane, bank conflicts, the splits and
the order of the folded write, the prefill's widened chunks and its mask-edge tiles."""

import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_attention_17_gb300", "csrc")

SOURCE = r'''
#include "e2m1_index.h"
using namespace pkv;
#define BOTH(name, call64, call128, ...) \
  extern "C" int name(int d, ##__VA_ARGS__) { return d == 128 ? call128 : call64; }
#define OF_D(name, expr) BOTH(name, (expr<64>()), (expr<128>()))
template <int D> int page_bytes_() { return E2m1Page<D>::kBytes; }
template <int D> int page_codes_() { return E2m1Page<D>::kCodes; }
template <int D> int row_codes_() { return E2m1Page<D>::kRowCodes; }
template <int D> int row_scales_() { return E2m1Page<D>::kRowScales; }
template <int D> int stage_bytes_() { return E2m1Stage<D>::kBytes; }
template <int D> int code_chunks_() { return E2m1Stage<D>::kCodeChunks; }
template <int D> int scale_lanes_() { return E2m1Stage<D>::kScaleLanes; }
OF_D(page_bytes, page_bytes_) OF_D(page_codes, page_codes_) OF_D(row_codes, row_codes_)
OF_D(row_scales, row_scales_) OF_D(stage_bytes, stage_bytes_) OF_D(code_chunks, code_chunks_)
OF_D(scale_lanes, scale_lanes_) OF_D(widen_rows, widen_step)
#define TWO(name, expr) \
  extern "C" int name(int d, int a, int b) { return d == 128 ? expr(128) : expr(64); }
#define STAGE_CODES(D) (E2m1Stage<D>::codes(a, b))
#define STAGE_SCALES(D) (E2m1Stage<D>::scales(a, b))
#define CODE_CHUNK(D) (E2m1Stage<D>::code_chunk(a, b))
#define SCALE_PAGE(D) (E2m1Stage<D>::scale_page(a))
#define SCALE_SOURCE(D) (E2m1Stage<D>::scale_source(a))
#define SCALE_DEST(D) (E2m1Stage<D>::scale_dest(a))
#define K_CODES(D) (k_codes_at<D>(a))
#define K_SCALES(D) (k_scales_at<D>(a))
#define V_CODES(D) (v_codes_at<D>(a, b))
#define V_SCALES(D) (v_scales_at<D>(a, b))
#define MERGE(D) (merge_chunk<D>(a, b))
#define W_BLOCK(D) (widen_block<D>(a))
#define W_ROW(D) (widen_row<D>(a))
TWO(stage_codes, STAGE_CODES) TWO(stage_scales, STAGE_SCALES) TWO(code_chunk, CODE_CHUNK)
TWO(scale_page, SCALE_PAGE) TWO(scale_source, SCALE_SOURCE) TWO(scale_dest, SCALE_DEST)
TWO(k_codes, K_CODES) TWO(k_scales, K_SCALES) TWO(v_codes, V_CODES) TWO(v_scales, V_SCALES)
TWO(merge, MERGE) TWO(w_block, W_BLOCK) TWO(w_row, W_ROW)
extern "C" int k_key(int lane) { return score_key(lane); }
extern "C" int v_key(int lane, int c) { return value_key(lane, c); }
extern "C" void range(int L, int n, int causal, int window, int i_first, int i_last, int splits,
                      int split, int* out) {
  const KeyRange r = key_range(L, n, causal, window, i_first, i_last, splits, split);
  out[0] = r.kv_lo; out[1] = r.kv_hi; out[2] = r.b_beg; out[3] = r.b_end;
  out[4] = new_keys_lo(L, n, r); out[5] = new_keys_hi(r);
}
static KeyRange blocks(int b_beg, int b_end) { return KeyRange{0, 0, b_beg, b_end}; }
extern "C" int pair(int b_beg, int warp, int warps, int k) { return pair_block(blocks(b_beg, 0), warp, warps, k); }
extern "C" int pairs(int b_beg, int b_end, int warp, int warps) { return warp_pairs(blocks(b_beg, b_end), warp, warps); }
extern "C" int waits(int b_beg, int new_lo, int warp, int warps) { return waiting_pair(blocks(b_beg, 0), new_lo, warp, warps); }
extern "C" int w_word(int block, int which) { return widen_word(block, which); }
extern "C" int w_to(int block, int row, int which) { return widen_to(block, row, which); }
extern "C" int w_half() { return kWidenHalf; }
extern "C" int edge(int kt, int ntk, int key0, int lim_first, int lo_last) { return edge_place(kt, ntk, key0, lim_first, lo_last); }
extern "C" int edge_tiles() { return kEdgeTiles; }
'''

LANES = range(32)


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("no host compiler")
    folder = tmp_path_factory.mktemp("e2m1_index")
    source, lib = folder / "index.cpp", folder / "index.so"
    source.write_text(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Wno-variadic-macros", "-fPIC", "-shared", "-I", CSRC,
                    str(source), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def ways(addresses, size):
    """Worst bank conflict of one phase of a shared-memory access of `size` bytes a lane."""
    per, worst = 128 // size, 1
    for p in range(0, len(addresses), per):
        banks = {}
        for a in addresses[p:p + per]:
            for b in range(0, size, 4):
                banks.setdefault((a + b) // 4 % 32, set()).add((a + b) // 4)
        worst = max([worst] + [len(x) for x in banks.values()])
    return worst


def test_the_kernels_take_their_indexes_from_this_file():
    """The expressions are called by name where the kernels used to spell them out."""
    decode = open(os.path.join(CSRC, "decode_e2m1.cu")).read()
    for name in ("score_key(lane)", "value_key(lane, c)", "value_key(q, c)", "k_codes_at<D>(lane)",
                 "k_scales_at<D>(lane)", "v_codes_at<D>(lane, c)", "v_scales_at<D>(lane, c)",
                 "merge_chunk<D>(rho", "key_range(L, n", "new_keys_lo(L, n, range.keys)",
                 "new_keys_hi(range.keys)", "pair_block(range.keys, warp", "warp_pairs(range.keys, warp",
                 "waiting_pair(range.keys, new_lo, warp", "Stage::codes(1, j)", "Stage::scales(1, j)",
                 "Stage::scale_dest(lane)", "Stage::scale_source(lane)", "Stage::code_chunk(lane, 0)"):
        assert name in decode, name
    prefill = open(os.path.join(CSRC, "prefill.cu")).read()
    for name in ("widen_block<D>(ct)", "widen_row<D>(ct)", "widen_step<D>()", "widen_word(b, 0)",
                 "widen_to(b, r0, 0)", "widen_to(b, r0, 1)", "edge_place(kt, ntk, key0"):
        assert name in prefill, name


def test_keys_of_both_contractions_agree(ix):
    assert sorted(ix.k_key(4 * g) for g in range(8)) == list(range(8))
    for lane in LANES:
        assert ix.k_key(lane) == ix.k_key(lane & ~3)
    for t4 in range(4):
        # the transposed score fragment holds the keys of MMA rows 2 t4, 2 t4 + 1, and + 8
        a, b = ix.k_key(4 * (2 * t4)), ix.k_key(4 * (2 * t4 + 1))
        for lane in range(t4, 32, 4):
            assert [ix.v_key(lane, c) for c in range(4)] == [a, b, a + 8, b + 8]
    assert sorted(ix.v_key(t, c) for t in range(4) for c in range(4)) == list(range(16))


@pytest.mark.parametrize("d", [64, 128])
def test_each_code_and_its_scale_is_read_by_one_lane(ix, d):
    row, srow = ix.row_codes(d), ix.row_scales(d)
    for at, scale_at, keys, width in (
            (ix.k_codes, ix.k_scales, 2, d // 8), (ix.v_codes, ix.v_scales, 4, d // 16)):
        seen = []
        for lane, c in itertools.product(LANES, range(keys)):
            if keys == 2:                                # the second key 8 rows on
                first, scale = at(d, lane, 0) + 8 * row * c, scale_at(d, lane, 0) + 8 * srow * c
            else:
                first, scale = at(d, lane, c), scale_at(d, lane, c)
            for byte in range(first, first + width):
                seen.append(byte)
                key, element = byte // row, 2 * (byte % row)
                # the scale it takes: its own row's, of the block of 16 (K at d 128: two blocks)
                assert scale + (element // 16 - 2 * (first % row) // 16) == key * srow + element // 16
        assert sorted(seen) == list(range(16 * row))


@pytest.mark.parametrize("d", [64, 128])
def test_bank_conflicts_of_the_stage_reads(ix, d):
    assert ways([ix.k_codes(d, lane, 0) for lane in LANES], d // 8) == (1 if d == 128 else 2)
    for c in range(4):
        assert ways([ix.v_codes(d, lane, c) for lane in LANES], d // 16) <= 2


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c", [0, 1])
def test_merge_rows_are_stored_without_conflicts_and_read_back(ix, d, c):
    for i in range(0, d // 16, 2):
        at = []
        for lane in LANES:
            row, g = 2 * (lane & 3) + c, lane >> 2
            at.append(row * d * 4 + ix.merge(d, row, g * (d // 32) + i // 2) * 16)
        assert ways(at, 16) == 1
    for row in range(16):
        assert sorted(ix.merge(d, row, chunk) for chunk in range(d // 4)) == list(range(d // 4))


@pytest.mark.parametrize("d", [64, 128])
def test_a_stage_is_copied_once(ix, d):
    codes, page = ix.page_codes(d), ix.page_bytes(d)
    assert page == 9 * d and ix.stage_bytes(d) == 4 * page
    copies = []
    for lane in LANES:
        for is_v, j, c in itertools.product(range(2), range(2), range(ix.code_chunks(d))):
            at = ix.code_chunk(d, lane, c)
            copies.append((ix.stage_codes(d, is_v, j) + at, (is_v, j, at)))
        if lane < ix.scale_lanes(d):
            p = ix.scale_page(d, lane, 0)
            copies.append((ix.scale_dest(d, lane, 0), (p // 2, p % 2, ix.scale_source(d, lane, 0))))
    assert sorted(to for to, _ in copies) == list(range(0, ix.stage_bytes(d), 16))
    assert len({source for _, source in copies}) == len(copies)
    for to, (is_v, j, at) in copies:
        assert to == (ix.stage_codes(d, is_v, j) + at if at < codes else ix.stage_scales(d, is_v, j) + at - codes)


@pytest.mark.parametrize("warps", [6, 8])
@pytest.mark.parametrize("splits", [1, 2, 5])
@pytest.mark.parametrize("causal", [0, 1])
def test_splits_partition_and_no_pair_is_loaded_before_its_new_rows(ix, warps, splits, causal):
    out = (ctypes.c_int * 6)()
    for length in (1, 5, 16, 17, 31, 33, 100, 640, 999):
        for n, window in itertools.product(range(1, min(4, length) + 1), (0, 1, 20, 200)):
            stored = set()
            for tile in ([(0, n - 1)], [(i, i) for i in range(n)]):      # one row tile, or one a token
                for i_first, i_last in tile:
                    blocks = []
                    want_lo = max(0, length - n + i_first - window + 1) if window else 0
                    want_hi = length - n + i_last + 1 if causal else length
                    for split in range(splits):
                        ix.range(length, n, causal, window, i_first, i_last, splits, split, out)
                        lo, hi, beg, end, new_lo, new_hi = out
                        assert (lo, hi) == (want_lo, want_hi)
                        blocks += range(beg, end)
                        stored |= set(range(new_lo, new_hi))
                        pairs = []
                        for w in range(warps):
                            npw = ix.pairs(beg, end, w, warps)
                            early = ix.waits(beg, new_lo, w, warps) if new_lo < new_hi else npw
                            for k in range(npw):
                                first = ix.pair(beg, w, warps, k)
                                pairs.append(first)
                                if k < early and new_lo < new_hi:        # loaded before the barrier
                                    assert (first + 2) * 16 <= new_lo
                        assert sorted(pairs) == list(range(beg, end, 2))
                    assert blocks == list(range(want_lo // 16, -(-want_hi // 16)))
            assert stored >= set(range(length - n, length))
            assert min(stored) >= length - n and max(stored) < length


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_widening_covers_a_tile_without_conflicts(ix, d):
    blocks, step, chunks = ix.row_scales(d), ix.widen_rows(d), {}
    for i in range(128 // step):
        for which in range(2):
            at = []
            for ct in range(64):
                b, r = ix.w_block(d, ct, 0), ix.w_row(d, ct, 0) + i * step
                word, to = ix.w_word(b, which), ix.w_to(b, r, which)
                # (the kernel steps from unit 0's place)
                assert to == ix.w_to(b, r - i * step, which) + i * step * 128
                # the chunk of 8 elements, where the MMA's 128-byte swizzle looks for it
                chunk = 2 * b + word
                assert to == chunk // 8 * ix.w_half() + r * 128 + ((chunk % 8) ^ (r % 8)) * 16
                assert (r, chunk) not in chunks
                chunks[r, chunk] = to
                at.append(to)
            assert ways(at[:32], 16) == 1 and ways(at[32:], 16) == 1
        reads = [(r // 16) * ix.page_bytes(d) + (r % 16) * ix.row_codes(d) + 8 * b
                 for b, r in ((ix.w_block(d, ct, 0), ix.w_row(d, ct, 0) + i * step) for ct in range(32))]
        assert ways(reads, 8) == 1
    assert sorted(chunks) == [(r, c) for r in range(128) for c in range(d // 8)]
    assert len(set(chunks.values())) == len(chunks)
    assert blocks * 16 == d


@pytest.mark.parametrize("causal", [0, 1])
def test_edge_tiles_have_places_of_their_own(ix, causal):
    half = ix.edge_tiles() // 2
    for pos0 in range(0, 700, 13):                       # first row's position
        for rows in (1, 100, 128, 200, 256):
            for window in (0, 128, 129, 300, 500):
                first = max(0, pos0 - window + 1) if window else 0
                kv_len = pos0 + rows
                base = first // 128
                ntk = -(-kv_len // 128) - base
                lim_first = pos0 + 1 if causal else kv_len
                lo_last = pos0 + rows - 1 - window + 1 if window else 0
                places = {}
                for kt in range(ntk):
                    key0 = (base + kt) * 128
                    place = ix.edge(kt, ntk, key0, lim_first, lo_last)
                    # every tile that some row does not see whole has a place
                    partial = key0 + 128 > lim_first or key0 < lo_last
                    assert (place >= 0) == partial
                    if place >= 0:
                        assert place < 2 * half and place not in places
                        places[place] = kt
                        # and is found again from its place
                        assert kt == (ntk - 1 - place if place < half else place - half)
