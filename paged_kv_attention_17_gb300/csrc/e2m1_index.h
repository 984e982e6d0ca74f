// Index arithmetic of the 4-bit cache's kernels: the page, which lane of a decode
// warp holds what, which keys and blocks a CTA takes, the order of the folded write,
// and the prefill's widening and mask-edge tiles.  Integers only, for the host too:
// tests/test_e2m1_index.py compiles this file and checks what the kernels use.
#pragma once

#if defined(__CUDACC__)
#define PKV_INDEX __host__ __device__ __forceinline__
#else
#define PKV_INDEX inline
#endif

namespace pkv {

PKV_INDEX int index_min(int a, int b) { return a < b ? a : b; }
PKV_INDEX int index_max(int a, int b) { return a > b ? a : b; }

// ---- the page of one (block, KV head) ----
constexpr int kQuant = 16;                               // elements per scale
constexpr int kPageTokens = 16;
template <int D>
struct E2m1Page {
  static constexpr int kRowCodes = D / 2;                // code bytes of a token row
  static constexpr int kRowScales = D / kQuant;          // scale bytes of a token row
  static constexpr int kCodes = kPageTokens * kRowCodes;
  static constexpr int kScales = kPageTokens * kRowScales;
  static constexpr int kBytes = kCodes + kScales;        // 9 D
};

// ---- a decode stage: two blocks' K codes, their V codes, K scales, V scales ----
template <int D>
struct E2m1Stage {
  using P = E2m1Page<D>;
  static constexpr int kPair = 2;                        // blocks per stage
  static constexpr int kScaleOff = 2 * kPair * P::kCodes;
  static constexpr int kBytes = 2 * kPair * P::kBytes;
  static PKV_INDEX int codes(int is_v, int j) { return (is_v * kPair + j) * P::kCodes; }
  static PKV_INDEX int scales(int is_v, int j) {
    return kScaleOff + (is_v * kPair + j) * P::kScales;
  }
  // Its copy, 16 bytes a lane: chunk c of the codes of a block and tensor, at
  // code_chunk in the page and behind codes(is_v, j); and one chunk of the scale areas
  // by the lanes below kScaleLanes, of page scale_page (K of both blocks, V of both),
  // from scale_source in it to scale_dest.
  static constexpr int kCodeChunks = P::kCodes / 512;
  static constexpr int kPageScaleLanes = P::kScales / 16;
  static constexpr int kScaleLanes = 2 * kPair * kPageScaleLanes;
  static PKV_INDEX int code_chunk(int lane, int c) { return lane * 16 + c * 512; }
  static PKV_INDEX int scale_page(int lane) { return lane / kPageScaleLanes; }
  static PKV_INDEX int scale_source(int lane) { return P::kCodes + (lane % kPageScaleLanes) * 16; }
  static PKV_INDEX int scale_dest(int lane) { return kScaleOff + lane * 16; }
};

// ---- a decode lane (g8 = lane / 4, t4 = lane % 4) ----
// K: the token rows score_key and score_key + 8 of a block, D / 4 elements from t4 D / 4
PKV_INDEX int score_key(int lane) {
  const int g8 = lane >> 2;
  return (g8 & 1) ? ((g8 >> 1) ^ 1) + 4 : g8 >> 1;
}
// V: the token rows value_key(lane, 0 .. 3), D / 8 elements from g8 D / 8
PKV_INDEX int value_key(int lane, int c) {
  const int t4 = lane & 3;
  return ((c & 1) ? (t4 ^ 1) + 4 : t4) + (c >> 1) * 8;
}
// where they begin, behind the codes (scales) of a block in a stage
template <int D>
PKV_INDEX int k_codes_at(int lane) {
  return score_key(lane) * E2m1Page<D>::kRowCodes + (lane & 3) * (D / 8);
}
template <int D>
PKV_INDEX int k_scales_at(int lane) {
  return score_key(lane) * E2m1Page<D>::kRowScales + (lane & 3) * (D / 64);
}
template <int D>
PKV_INDEX int v_codes_at(int lane, int c) {
  return value_key(lane, c) * E2m1Page<D>::kRowCodes + (lane >> 2) * (D / 16);
}
template <int D>
PKV_INDEX int v_scales_at(int lane, int c) {
  return value_key(lane, c) * E2m1Page<D>::kRowScales + (lane >> 2) * D / 128;
}
// where a merge row keeps a 16-byte chunk
template <int D>
PKV_INDEX int merge_chunk(int row, int chunk) {
  return chunk ^ (D == 128 ? (row >> 1) & 3 : ((row >> 1) & 1) | (row & 4));
}

// ---- the keys [kv_lo, kv_hi) that the rows of tokens i_first .. i_last of a request
// (n new tokens, L keys) see, and the blocks [b_beg, b_end) of one split of them ----
struct KeyRange {
  int kv_lo, kv_hi, b_beg, b_end;
};
PKV_INDEX KeyRange key_range(int L, int n, int causal, int window, int i_first, int i_last,
                             int splits, int split) {
  KeyRange r;
  r.kv_hi = causal ? L - n + i_last + 1 : L;
  r.kv_lo = window > 0 ? index_max(0, L - n + i_first - window + 1) : 0;
  const int blk_lo = r.kv_lo / kPageTokens;
  const int nb = (r.kv_hi + kPageTokens - 1) / kPageTokens - blk_lo;
  const int per = (nb + splits - 1) / splits;
  r.b_beg = blk_lo + index_min(nb, split * per);
  r.b_end = blk_lo + index_min(nb, (split + 1) * per);
  return r;
}
// the new tokens' keys [lo, hi) among them: what the folded write of that CTA stores
PKV_INDEX int new_keys_lo(int L, int n, const KeyRange& r) {
  return index_max(L - n, index_max(r.kv_lo, r.b_beg * kPageTokens));
}
PKV_INDEX int new_keys_hi(const KeyRange& r) {
  return index_min(r.kv_hi, r.b_end * kPageTokens);
}
// Pair k of a warp begins at this block, and its first `waiting_pair` pairs hold no
// key from new_lo on (they are loaded before the write).
PKV_INDEX int pair_block(const KeyRange& r, int warp, int warps, int k) {
  return r.b_beg + 2 * (warp + k * warps);
}
PKV_INDEX int warp_pairs(const KeyRange& r, int warp, int warps) {
  const int npairs = (r.b_end - r.b_beg + 1) / 2;
  return npairs > warp ? (npairs - warp - 1) / warps + 1 : 0;
}
PKV_INDEX int waiting_pair(const KeyRange& r, int new_lo, int warp, int warps) {
  return (new_lo / kPageTokens - r.b_beg - 2 * warp) / (2 * warps);
}

// ---- prefill: widening of a 128-key tile by 64 threads ----
constexpr int kWidenHalf = 16384;                        // bytes of 64 f16 columns of the tile
// Unit i of thread ct is one scale block of one key row.
template <int D>
PKV_INDEX int widen_block(int ct) {
  return ct % E2m1Page<D>::kRowScales;
}
template <int D>
PKV_INDEX int widen_row(int ct) {                        // of unit 0
  return ct / E2m1Page<D>::kRowScales;
}
template <int D>
PKV_INDEX int widen_step() {                             // rows from a unit to the next: 8 or 16
  return 64 / E2m1Page<D>::kRowScales;
}
// Its two words of 8 codes become two 16-byte chunks.  Store `which` (0, 1) takes word
// widen_word, to widen_to in the tile (128-byte rows, chunk c of row r at c ^ (r % 8)).
// The blocks of the second column half store their words the other way round.
PKV_INDEX int widen_word(int block, int which) { return (block >> 2) ^ which; }
PKV_INDEX int widen_to(int block, int row, int which) {
  return (block >> 2) * kWidenHalf + row * 128 +
         (((2 * (block & 3) + widen_word(block, which)) ^ (row & 7)) << 4);
}

// ---- prefill: tiles that some row of a unit does not see whole ----
// A unit's rows are at most 256 consecutive positions: 3 tiles of 128 keys at either
// end.  The place of tile kt (of ntk, from key0) among them, -1 if every row sees all
// of its keys below lim_first (the first row's limit) and from lo_last (the last row's
// window start).
constexpr int kEdgeTiles = 6;
PKV_INDEX int edge_place(int kt, int ntk, int key0, int lim_first, int lo_last) {
  if (key0 + 128 > lim_first && ntk - 1 - kt < kEdgeTiles / 2) return ntk - 1 - kt;
  if (key0 < lo_last && kt < kEdgeTiles / 2) return kEdgeTiles / 2 + kt;
  return -1;
}

}  // namespace pkv
