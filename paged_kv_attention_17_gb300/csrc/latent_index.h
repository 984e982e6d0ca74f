// How a batch's key tiles are dealt out in absorbed latent attention.  Integers only,
// for the host too: tests/test_latent_index.py compiles this file and checks what the
// kernel uses.
//
// A request's (token, head) rows are cut into units of 64.  The unit of rows 64 j .. 64 j
// + 63 has as many key tiles of 64 as its last row sees.  Every unit of a request is given
// the same cost, kUnitCost for its start and end and the mean of its first and last unit's
// tiles, and the units are taken in the order first, last, second, last but one, ..., so that
// neighbours together have about that many, and a position in the batch's total cost is
// found without adding units up.  Block c of the grid takes the positions [c per, (c + 1)
// per); where that cuts a unit, its tiles are cut in the same proportion.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define PKV_LATENT_INDEX __host__ __device__ __forceinline__
#else
#define PKV_LATENT_INDEX inline
#endif

namespace pkv {

constexpr int kUnitRows = 64;                    // rows of a unit
constexpr int kTileKeys = 64;                    // keys of a tile
// Tiles that a unit's start and end take as long as.  With 1, 2, 3, 4 and 6, in us: 16 requests of 6
// units on 100 to 9000 keys 104.6, 99.0, 97.5, 100.4, 101.8; 32 requests of 2 units on 200 to 3000
// keys 44.4, 39.9, 41.2, 42.0, 43.2; 256 requests of one unit on 200 to 900 keys 47.9, 48.2, 49.2,
// 50.6, 52.8; 64 on 512 to 4096 keys 48.5, 48.4, 48.6, 49.0, 50.3; 4 requests of 75 units 106.6 with
// any.  2 and 3 are within 3% of each other everywhere; 3 does better where it saves most.
constexpr int kUnitCost = 3;

// a / b (b > 0) by a 32-bit division where that will do: the 64-bit one is a long call.
PKV_LATENT_INDEX int64_t quotient(int64_t a, int64_t b) {
  const uint64_t x = static_cast<uint64_t>(a), y = static_cast<uint64_t>(b);
  return ((x | y) >> 32) == 0
             ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y))
             : static_cast<int64_t>(x / y);
}

// rows = n * hq < 2^31
struct LatentRequest {
  int rows, units, cost;                         // 0 units: nothing to do
  int lead, full, hq, causal;                    // keys that row 0 and the last row see
  PKV_LATENT_INDEX int row_limit(int row) const {
    return causal ? lead + static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(hq))
                  : lead;
  }
  // keys that the unit's last row sees (most requests are one unit: no division)
  PKV_LATENT_INDEX int limit(int j) const {
    return j + 1 >= units ? full : row_limit(j * kUnitRows + (kUnitRows - 1));
  }
  PKV_LATENT_INDEX int tiles(int j) const {
    return static_cast<int>((static_cast<uint32_t>(limit(j)) + kTileKeys - 1) / kTileKeys);
  }
};

// valid: a request that the kernel can attend (lengths and rows within their bounds).
PKV_LATENT_INDEX LatentRequest latent_request(bool valid, int n, int L, int hq, int causal) {
  LatentRequest r;
  r.lead = causal ? L - n + 1 : L;
  r.full = L;
  r.hq = hq;
  r.causal = causal;
  r.rows = valid ? n * hq : 0;
  r.units = static_cast<int>((static_cast<uint32_t>(r.rows) + kUnitRows - 1) / kUnitRows);
  r.cost = 0;
  if (r.units > 0) {
    const int last = r.tiles(r.units - 1);
    r.cost = kUnitCost + (causal && r.units > 1 ? (r.tiles(0) + last + 1) / 2 : last);
  }
  return r;
}

// the unit that the u-th place of a request's order holds
PKV_LATENT_INDEX int unit_at(int u, int units) { return u % 2 == 0 ? u / 2 : units - 1 - u / 2; }

// positions a block takes
PKV_LATENT_INDEX int64_t positions_per_block(int64_t total, int blocks, int64_t least) {
  const int64_t per = quotient(total + blocks - 1, blocks);
  return per > least ? per : least;
}

// A block's walk over its pieces.  Start it at position v of the total, at place u and
// offset o (of cost) in request r; next() gives a piece of the current request, false once
// the request's units are used up (give it the next request) or at the end (v == end).
struct LatentPiece {
  int unit;                                      // within the request
  int tile0, tile1;                              // key tiles [tile0, tile1), maybe none
  bool first, last;                              // holds the unit's start, its end
  int rest;                                      // of its cost, for later blocks
};
// pieces of a unit that a block begins and leaves `rest` of
PKV_LATENT_INDEX int pieces_of(int rest, int64_t per) {
  return rest <= per ? 2 : 1 + static_cast<int>(quotient(rest + per - 1, per));
}
// the tiles of a unit of `tiles` that lie before offset o of its cost
PKV_LATENT_INDEX int tiles_before(int o, int tiles, int cost) {
  const int past = o > kUnitCost ? o - kUnitCost : 0, span = cost - kUnitCost;
  return span == tiles ? past
                       : static_cast<int>(quotient(static_cast<int64_t>(past) * tiles, span));
}
struct LatentWalk {
  int64_t v, end;
  int u, o;
  PKV_LATENT_INDEX bool next(const LatentRequest& r, LatentPiece& p) {
    if (v >= end || u >= r.units) return false;
    const int rest = r.cost - o;
    const int take = rest < end - v ? rest : static_cast<int>(end - v);
    p.unit = unit_at(u, r.units);
    const int tiles = r.tiles(p.unit);
    p.first = o == 0;
    p.last = take == rest;
    p.tile0 = p.first ? 0 : tiles_before(o, tiles, r.cost);
    p.tile1 = p.last ? tiles : tiles_before(o + take, tiles, r.cost);
    p.rest = rest - take;
    v += take;
    o = 0;
    ++u;
    return true;
  }
};

// What is done about the block at place b of a unit's keys, which end in place `blocks` - 1:
// entry is what the block table holds there.  By the place, as an entry may have any value.
enum class Page { kLoad, kBehind, kBad };
PKV_LATENT_INDEX Page page_of(int b, int blocks, int entry, int64_t num_blocks) {
  if (b >= blocks) return Page::kBehind;
  return entry >= 0 && entry < num_blocks ? Page::kLoad : Page::kBad;
}

// Time, beyond a single wait's, that a piece of so many tiles may take at most: a tile takes 1.0
// to 2.0 us as it streams, and this allows ten times that.
PKV_LATENT_INDEX uint64_t piece_limit_ns(int tiles) { return static_cast<uint64_t>(tiles) * 20000; }

// Partials: block c keeps the piece that begins inside a unit in slot 2 c, the piece that
// a later block goes on with in slot 2 c + 1.
PKV_LATENT_INDEX int piece_slot(int block, bool first) { return 2 * block + (first ? 1 : 0); }

}  // namespace pkv
