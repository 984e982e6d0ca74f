// Latent attention in the absorbed form, on the 5th-generation tensor cores (tcgen05 +
// TMEM + TMA).
//
// All heads of a token attend the same cached rows [c | r] of 512 + 64 elements, whose
// first 512 are the values too: S = Q C^T, P = softmax(S), O = P C[:, :512].  "Inside the
// engine ...", sections "Never materialise the TxT matrix" (online softmax over key
// tiles), "Attention over a block table ..." (rows gathered block by block) and "Prefill
// has a full grid; decode at batch 1 has almost none" (any split of the keys, merged).
//
// A unit is 64 (token, head) rows of a request, consecutive in memory; a tile is 64 keys.
// A key row is read once for both products:
//   S (64 x 64) = Q C^T   A = Q, B = C, both K-major in shared memory (9 slabs of 64
//                         elements, 128-byte swizzle), 36 MMAs of M 64, N 64;
//   O^T (512 x 64) += C^T P^T   A = C^T, the same slabs read MN-major, B = P (64 x 64,
//                         K-major), 16 MMAs of M 128, N 64.
// O is held transposed, since 64 x 512 fp32 with 64 rows a lane half would be all of
// TMEM: 4 x 64 columns of 128 lanes, beside two buffers of S (64 columns each, rows 16 w ..
// 16 w + 15 in the first 16 lanes of quarter w, where M = 64 puts them).
//
// Block: warps 0-3 and 4-7 softmax of the two halves of a tile's keys, and output; 8-11
// load keys, each one cache block of every tile (a thread that waits, announces and issues
// takes 500 cycles a load of 18 KB, so one would bring 34 bytes a cycle; four bring the 71
// that the copy engine gives); 12 issues the MMAs, whichever product is ready, so that the
// softmax of one tile runs beside the products of another; 13 works out the block's pieces
// ahead of the others and loads their queries.  Two stages of 64 keys (72 KB each, beside 72
// KB of queries); a stage's halves are freed one after the other as O goes on.
// The grid is one block an SM; each takes an equal run of the batch's tiles
// (latent_index.h), so that ragged contexts, few requests and many heads all fill the
// machine, and writes a unit that it holds whole itself, the others' pieces as fp32
// partials for the merge kernel.
//
// The running maximum is a reference that moves only when a row's maximum is 8 log2 units
// above it: p <= 2^8, and O is rescaled rarely.
//
// A hidden key's p is 0, but 0 times a NaN value is a NaN: in the tiles that cross a row's
// limit, keys behind the unit's last one are zeroed, and so is a key that some of the unit's
// rows do not see and whose scores are non-finite for all of them (any key with a NaN or an
// infinity is).  The rows that do see it are NaN by its score, unless that is -inf: then, as in
// every other tile, only the elements that 0 times an infinity makes so (spoil).
//
// What bounds it.  HBM where a key meets few rows; from about 64 rows a key, shared memory: a
// tile of 64 keys and 64 rows is 36 MMAs that read 4 KB each and 16 that read 6 KB, beside 72
// KB that the copy engine writes, 2500 cycles at 128 bytes a cycle; it takes about 2900.
// (Counted, of all active cycles of the 16 requests below, start and end among them: the tensor
// cores read shared memory in 53%, the warps use it in 6%; the copy engine's bytes are another
// 16%.  A tile of 128 rows would halve the reads a row, but its queries leave no room for
// two stages of keys.)  Few tiles a block: the way to the first scores, 6 us (lengths, table and keys
// are fetched one after the other), and the merge's launch and its fetch, 5 us.
// Measured: 1 request of 8192 keys, 16 heads, 14.3 us; 64 of 512 to 4096 keys, 32 heads, 43.3 us
// (153 MB, 3.5 TB/s); 2 of 131000, 64 heads, 69 us (302 MB, 4.4 TB/s); 16 of three tokens and
// 100 to 9000 keys, 128 heads, 101 us (0.64 PFLOP/s).
#include <algorithm>

#include "device_set.h"
#include "latent.cuh"
#include "latent_index.h"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 448;
constexpr int kSoftmax = 256;                    // threads of warps 0-7
constexpr int kLoadWarp = 8, kMmaWarp = 12, kPlanWarp = 13;
constexpr int kJobs = 4;                         // pieces worked out ahead
// Requests whose lengths one warp adds up, while the others go on: 1 request 14.2 us, against
// 14.7 with the whole block.  (64 requests: 42.6 and 42.7; beyond, a lane would read many.)
constexpr int kFewRequests = 128;
constexpr int kStages = 2;
constexpr int kSlabs = kLatentRow / 64;          // 9 column slabs of 64 elements (128 bytes)
constexpr int kSlab = 64 * 128;                  // queries: [slab][64 rows][128 bytes]
// keys: [8-key group][slab][8 rows][128 bytes], as one load of 8 rows leaves them
constexpr int kGroup = kSlabs * 1024;
constexpr int kPart = 2 * kGroup;                // a cache block's 16 keys
constexpr int kParts = kTileKeys / kBlock;       // 4
constexpr int kTile = kParts * kPart;
constexpr int kQueries = kSlabs * kSlab;
constexpr int kOffTiles = kQueries;
constexpr int kOffP = kOffTiles + kStages * kTile;
constexpr int kOffBars = kOffP + kSlab;
// full[stage], empty[stage][half], s[buffer], q_full, q_empty, p[half], job_full[], job_empty[]
constexpr int kBars = kStages + kStages * 2 + 2 + 2 + 2 + 2 * kJobs;
constexpr int kOffMisc = (kOffBars + kBars * 8 + 15) / 16 * 16;
// factors[64], tops[half][64], bad[2], tmem
constexpr int kOffStart = kOffMisc + 3 * kUnitRows * 4 + 16;
constexpr int kOffJobs = kOffStart + 192;        // (start, then the warps' sums)
constexpr int kSmem = kOffJobs + kJobs * 64 + 1024;
static_assert(kSmem <= 232448, "shared memory of the absorbed kernel");
static_assert(kOffTiles % 1024 == 0 && kOffP % 1024 == 0 && kOffMisc % 16 == 0 && kOffStart % 16 == 0 &&
                  kOffJobs % 16 == 0, "alignment of what lies in shared memory");
constexpr int kTmemCols = 512;
constexpr int kColO = 0, kColS = 256;
constexpr float kSlack = 8.f;
constexpr float kNoKeys = INFINITY;              // for the log-sum-exps of a piece without tiles
// Tiles a block takes at least (it matters where there are few).  With 1 (more pieces to merge),
// 2, 3 and 4, in us: 1 request of 1000 keys, 16 heads, 12.4, 12.4, 14.8, 15.4; of 8192 keys 15.0,
// 14.8, 15.7, 16.3, with 128 heads 18.8, 18.8, 20.3, 20.6; of 40000 keys 23.1, 22.9, 23.1, 23.0;
// 4 of 4000 keys 15.6, 15.6, 17.1, 17.6; 8 of 300 to 2000, 32 heads, 18.7, 18.7, 17.2, 17.7.
constexpr int kLeastPositions = 2;
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeBatch = 16;                  // pieces a thread has in flight
constexpr int kMostBlocks = 255;                 // (a piece's weight has a lane of a warp)
static_assert(kMostBlocks <= kMergeThreads && kMostBlocks + 1 <= 32 * kMergeWarps,
              "units and weights of the merge");

struct alignas(16) Unsplit {                     // a unit that block c begins and others end
  int64_t row;                                   // its first (token, head) row
  int rows, pieces;                              // 0 pieces: none
};

struct Layout {                                  // of the workspace
  size_t lse, units, bytes;
};
__host__ __device__ inline Layout layout(int blocks) {
  Layout l;
  l.lse = static_cast<size_t>(blocks) * 2 * kUnitRows * kLatent * sizeof(float);
  l.units = l.lse + static_cast<size_t>(blocks) * 2 * kUnitRows * sizeof(float);
  l.bytes = l.units + static_cast<size_t>(blocks) * sizeof(Unsplit);
  return l;
}
// a row's log2 log-sum-exps lie together: the merge reads those of a row's pieces
__device__ __forceinline__ int lse_at(int row, int slot, int blocks) { return row * 2 * blocks + slot; }

// mbar_wait by polling: the suspended wait wakes up some hundred cycles late.
__device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity,
                                     unsigned long long limit_ns = kWaitLimitNs) {
  unsigned long long t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (mbar_ready(bar, parity)) return true;
    if ((i & 255) == 255) {
      const unsigned long long t = globaltimer();
      if (t0 == 0) t0 = t;
      else if (t - t0 > limit_ns) return false;
    }
  }
}

// Request r, with no units where its lengths are out of bounds (told once).
__device__ __forceinline__ LatentRequest request(const LatentArgs& a, int r, int& q0, bool tell) {
  q0 = __ldg(a.qsl + r);
  const int q1 = __ldg(a.qsl + r + 1), L = __ldg(a.seq_lens + r);
  const int64_t n = static_cast<int64_t>(q1) - q0;
  const bool valid = q0 >= 0 && n >= 0 && q1 <= a.num_tokens && n <= L && n <= a.max_query_len &&
                     L <= (1 << 30) && L <= static_cast<int64_t>(a.max_blocks_per_seq) * kBlock;
  if (tell && (!valid || (r == 0 && q0 != 0))) raise_flag(a.flag, PKV_FLAG_BAD_LENGTHS);
  return latent_request(valid, static_cast<int>(valid ? n : 0), L, a.hq, a.causal);
}

struct Start {                                   // a block's first position
  int64_t v, end, per;
  int r, u, o, some, q0;
  LatentRequest request;                         // r's
};
static_assert(sizeof(Start) + (kThreads / 32) * 8 <= 192, "the block's start in shared memory");

// Where block blockIdx.x starts: each of T threads (a warp, or the block) sums the costs of a
// run of requests, and the one in whose run the block's first position lies looks for it
// there.
template <int T>
__device__ __forceinline__ void find_start(const LatentArgs& a, Start* s, int64_t* sums) {
  const int tid = T == 32 ? threadIdx.x & 31 : threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (a.num_seqs + T - 1) / T;
  const int r0 = min(tid * run, a.num_seqs), r1 = min(r0 + run, a.num_seqs);
  int64_t sum = 0;
  int q0;
  LatentRequest x;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    x = request(a, r, q0, blockIdx.x == 0);
    sum += static_cast<int64_t>(x.units) * x.cost;
  }
  int64_t upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  int64_t total = __shfl_sync(0xffffffffu, upto, 31), before = upto - sum;
  if (tid == 0) s->some = 0;
  if constexpr (T > 32) {
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
  } else {
    __syncwarp();
  }
  const int64_t per = positions_per_block(total, gridDim.x, kLeastPositions);
  const int64_t v = blockIdx.x * per;
  if (v >= before && v < before + sum) {
    int64_t at = before;
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      if (run > 1) x = request(a, r, q0, false);
      const int64_t cost = static_cast<int64_t>(x.units) * x.cost;
      if (v < at + cost) {
        s->v = v;
        s->end = min(v + per, total);
        s->per = per;
        s->u = static_cast<int>(quotient(v - at, x.cost));
        s->o = static_cast<int>((v - at) - static_cast<int64_t>(s->u) * x.cost);
        s->r = r;
        s->q0 = q0;
        s->request = x;
        s->some = 1;
        break;
      }
      at += cost;
    }
  }
  if constexpr (T > 32) __syncthreads();
  else __syncwarp();
}

// A piece as the roles need it.
struct Job {
  int row0, rows;                                // (token, head) rows; 0 rows: no more pieces
  int tile0, tile1;
  int request, blocks;                           // cache blocks of the unit's keys
  int lead, first_row;                           // keys of the request's row 0; the unit's first row
  int first, last;                               // holds the unit's start, its end
  int pieces;                                    // of the unit, where it begins here
};
static_assert(sizeof(Job) <= 64, "pieces in shared memory");

// NaN in the elements of a piece's output (bf16 rows, or fp32 partials) that a key of [key0,
// key1) spoils, which some of its rows see and others do not: those where the key holds an
// infinity or a NaN, of the rows that see it.  The key weighs 0 there.  (Rare, and so out of the
// way: a thread looks its two dims up in the cache.)
template <typename T>
__device__ __noinline__ void spoil(T* to, T nan, const __nv_bfloat16* cache, const int32_t* table,
                                   int64_t num_blocks, int hq, int lead, int first_row, int rows,
                                   int key0, int key1, int dim0) {
#pragma unroll 1
  for (int key = key0; key < key1; ++key) {
    const int block = __ldg(table + key / kBlock);
    if (block < 0 || block >= num_blocks) continue;
    const __nv_bfloat16* x = cache + (static_cast<int64_t>(block) * kBlock + key % kBlock) * kLatentRow;
    // (row i of the request sees the keys below lead + i / hq)
    const int64_t from = static_cast<int64_t>(key + 1 - lead) * hq - first_row;
#pragma unroll 1
    for (int dim = dim0; dim < kLatent; dim += 256) {
      if ((__bfloat16_as_ushort(x[dim]) & 0x7F80u) != 0x7F80u) continue;
#pragma unroll 1
      for (int row = from > 0 ? static_cast<int>(from) : 0; row < rows; ++row)
        to[static_cast<int64_t>(row) * kLatent + dim] = nan;
    }
  }
}

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap cmap, const LatentArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBars);   // [stage]
  uint64_t* empty = full + kStages;              // [stage][half]: O has taken these keys
  uint64_t* bar_s = empty + kStages * 2;         // [buffer]: S is complete
  uint64_t* q_full = bar_s + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* bar_p = q_empty + 1;                 // [half]: P is stored, O rescaled
  uint64_t* job_full = bar_p + 2;
  uint64_t* job_empty = job_full + kJobs;
  float* factor = reinterpret_cast<float*>(smem + kOffMisc);       // O's rows are scaled by
  float* tops = factor + kUnitRows;              // [half][row]
  uint32_t* bad = reinterpret_cast<uint32_t*>(tops + 2 * kUnitRows);
  uint32_t* tmem = bad + 2;
  Start* start = reinterpret_cast<Start*>(smem + kOffStart);
  int64_t* sums = reinterpret_cast<int64_t*>(start + 1);
  Job* jobs = reinterpret_cast<Job*>(smem + kOffJobs);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Layout ws = layout(gridDim.x);
  uint8_t* const wsp = static_cast<uint8_t*>(a.workspace);

  // (nothing here depends on the kernel before)
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (uint64_t* b = full; b < full + kBars; ++b)
      // (a piece is released by 4 loading warps, the MMAs and 8 softmax warps)
      mbar_init(b, b < empty || b == bar_p || b == bar_p + 1 ? 4 : b >= job_empty ? 13 : 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(tmem, kTmemCols);
  if (warp == kLoadWarp && lane == 0) tma_prefetch_desc(&cmap);
  if (warp == kPlanWarp && lane == 0) tma_prefetch_desc(&qmap);
  if (warp == 0) {
    // (a line a thread of the block table, if that covers it, while the lengths are read)
    const int64_t entries = static_cast<int64_t>(a.num_seqs) * a.max_blocks_per_seq;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * 32;
    if (entries <= static_cast<int64_t>(gridDim.x) * 1024 && at < entries) prefetch_l2(a.block_table + at);
  }
  tc::fence_before();
  pdl_wait_primary();
  // (the planning warp finds the start of a batch of few requests by itself)
  const bool alone = a.num_seqs <= kFewRequests;
  if (alone) __syncthreads();
  else find_start<kThreads>(a, start, sums);
  tc::fence_after();
  const uint32_t tbase = *tmem;
  uint32_t it = 0;                               // tiles so far
  bool ok = true;
  // job k, once it is there
  auto job_ready = [&](uint32_t k) { return poll(&job_full[k % kJobs], (k / kJobs) & 1); };

  if (warp == kPlanWarp) {
    // ================= pieces, queries (one lane) =================
    if (alone) find_start<32>(a, start, sums);
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_first();
      LatentWalk w{0, 0, 0, 0};                  // (a block without positions has no pieces)
      int64_t per = 1;
      int r = 0, q0 = 0;
      LatentRequest x = latent_request(false, 0, 0, 1, 0);
      LatentPiece p;
      if (start->some) {
        w = LatentWalk{start->v, start->end, start->u, start->o};
        per = start->per;
        r = start->r;
        q0 = start->q0;
        x = start->request;
      }
      uint32_t units = 0;
      int tiles = 0;                             // of the piece whose queries are loaded
      for (uint32_t k = 0; ok; ++k) {
        bool more = w.next(x, p);
        while (!more && w.v < w.end && r + 1 < a.num_seqs) {
          x = request(a, ++r, q0, false);
          w.u = 0;
          w.o = 0;
          more = w.next(x, p);
        }
        if (k >= kJobs) ok = poll(&job_empty[k % kJobs], (k / kJobs - 1) & 1);
        if (!ok) break;
        Job& j = jobs[k % kJobs];
        j.rows = 0;
        if (more) {
          j.first_row = p.unit * kUnitRows;
          j.row0 = q0 * a.hq + j.first_row;
          j.rows = min(kUnitRows, x.rows - j.first_row);
          j.tile0 = p.tile0;
          j.tile1 = p.tile1;
          j.request = r;
          j.blocks = (x.limit(p.unit) + kBlock - 1) / kBlock;
          j.lead = x.lead;
          j.first = p.first;
          j.last = p.last;
          j.pieces = 0;
          if (p.first && !p.last) j.pieces = pieces_of(p.rest, per);
        }
        mbar_arrive(&job_full[k % kJobs]);
        if (!more) break;
        if (p.tile0 >= p.tile1) continue;
        // (this one wait is as long as a piece)
        if (units > 0) ok = poll(q_empty, (units - 1) & 1, kWaitLimitNs + piece_limit_ns(tiles));
        if (!ok) break;
        tiles = p.tile1 - p.tile0;
        mbar_arrive_expect_tx(q_full, kQueries);
        for (int s = 0; s < kSlabs; ++s)
          tc::load_2d(smem + s * kSlab, &qmap, q_full, s * 64, j.row0, policy);
        ++units;
      }
      if (!ok) {
        raise_flag(a.flag, PKV_FLAG_TIMEOUT);
        if (units > 0) poll(q_full, (units - 1) & 1);
      }
    }
  } else if (warp >= kLoadWarp && warp < kMmaWarp) {
    // ================= keys: block g of every tile (one lane) =================
    if (lane == 0) {
      const int g = warp - kLoadWarp;
      const uint64_t policy = l2_policy_evict_last();
      for (uint32_t k = 0; ok; ++k) {
        if (!(ok = job_ready(k))) break;
        const Job j = jobs[k % kJobs];
        mbar_arrive(&job_empty[k % kJobs]);
        if (j.rows == 0) break;
        const int32_t* table = a.block_table + static_cast<int64_t>(j.request) * a.max_blocks_per_seq;
        const int blocks = min(j.blocks, j.tile1 * kParts);
        // (-1 behind the keys, where the table is not looked at)
        auto entry = [&](int b) { return b < blocks ? __ldg(table + b) : -1; };
        // the tiles after the next are brought into L2 meanwhile: more in flight than shared
        // memory has room for (not before the block's first tile has landed: every block
        // waits for that one)
        auto hint = [&](int e) {
          if (e >= 0 && e < a.num_blocks)
            bulk_prefetch_l2(a.cache + static_cast<int64_t>(e) * (kBlock * kLatentRow), kPart);
        };
        int b = j.tile0 * kParts + g;
        int now = entry(b), next = entry(b + kParts);
#pragma unroll 1
        for (; b < j.tile1 * kParts; b += kParts, ++it) {
          const int later = entry(b + 2 * kParts);
          const int st = it % kStages;
          if (it == kStages) {
            if (!(ok = poll(&full[0], 0))) break;
            hint(now);
            hint(next);
          }
          if (it >= kStages && !(ok = poll(&empty[st * 2 + g / 2], ((it / kStages) - 1) & 1))) break;
          const Page page = page_of(b, blocks, now, a.num_blocks);
          if (page == Page::kLoad) {
            uint8_t* to = smem + kOffTiles + st * kTile + g * kPart;
            mbar_arrive_expect_tx(&full[st], kPart);
            tma_load_3d(to, &cmap, &full[st], 0, now * kBlock, 0, policy);
            tma_load_3d(to + kGroup, &cmap, &full[st], 0, now * kBlock + 8, 0, policy);
          } else {
            // behind the keys (its scores are hidden and O does not take it), or no block of
            // the cache (the row is unspecified)
            if (page == Page::kBad) raise_flag(a.flag, PKV_FLAG_BAD_BLOCK);
            mbar_arrive(&full[st]);
          }
          if (it >= kStages) hint(later);
          now = next;
          next = later;
        }
      }
      if (!ok) {
        // (given up: the loads that were issued land before the block may end)
        raise_flag(a.flag, PKV_FLAG_TIMEOUT);
        for (uint32_t t = it >= kStages ? it - kStages : 0; t < it; ++t)
          poll(&full[t % kStages], (t / kStages) & 1);
      }
    }
  } else if (warp == kMmaWarp) {
    // ================= MMAs (the whole warp: see mma_ss) =================
    constexpr uint32_t id_s = tc::instr_desc(kUnitRows, kTileKeys, false, false);
    const uint64_t dq = tc::smem_desc(smem_u32(smem), 16, 1024);
    const uint64_t dk = tc::smem_desc(smem_u32(smem + kOffTiles), 16, kGroup);
    const uint64_t dv = tc::smem_desc(smem_u32(smem + kOffTiles), 1024, kGroup);
    const uint64_t dp = tc::smem_desc(smem_u32(smem + kOffP), 16, 1024);
    auto ready = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_ready(bar, parity)) != 0;
    };
    // Two walks over the pieces: the scores' runs up to two tiles ahead of the values' (S
    // has two buffers, read before P is stored).  Whichever is ready goes next.
    uint32_t is = 0, units = 0;                            // scores issued; units begun
    uint32_t job_s = 0, job_o = 0;                         // the walks' next pieces
    int left_s = 0, left_o = 0, parts_o = 0;               // tiles left of their pieces, blocks
    bool end_s = false, begins_s = false, begins_o = false;
    uint32_t id_o = 0;
    unsigned long long since = 0;
    uint32_t idle = 0;
    while (true) {
      if (left_o == 0 && job_o < job_s) {                  // (seen by the other walk)
        const Job& j = jobs[job_o % kJobs];
        const int rows = j.rows;
        if (rows > 0) {
          left_o = j.tile1 - j.tile0;
          parts_o = min(j.blocks, j.tile1 * kParts) - j.tile0 * kParts;
          // (O for as many rows as there are, of 16, 32 and 64)
          id_o = tc::instr_desc(128, rows <= 16 ? 16 : rows <= 32 ? 32 : 64, true, false);
          begins_o = true;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_empty[job_o % kJobs]);
        ++job_o;
        if (rows == 0) break;
        continue;
      }
      bool moved = false;
      if (left_o > 0 && it < is && ready(&bar_p[0], it & 1)) {
        // O of a tile whose P is stored: block by block, halves freed as it goes
        tc::fence_after();
        const int st = it % kStages;
        const uint64_t tile = dv + (static_cast<uint64_t>(st * kTile) >> 4);
#pragma unroll
        for (int g = 0; g < kParts; ++g) {
          if (g == kParts / 2) {
            ok = __all_sync(0xffffffffu, poll(&bar_p[1], it & 1)) != 0;
            tc::fence_after();
          }
          if (g < parts_o) {
#pragma unroll
            for (int m = 0; m < 4; ++m)
              tc::mma_ss(tbase + kColO + m * kUnitRows,
                         tile + (static_cast<uint64_t>(g * kPart + 2 * m * 1024) >> 4),
                         dp + (static_cast<uint64_t>(g * 32) >> 4), id_o, !begins_o || g > 0);
          }
          if (g % 2 == 1) tc::commit(&empty[st * 2 + g / 2]);
        }
        if (!ok) break;
        begins_o = false;
        ++it;
        --left_o;
        parts_o -= kParts;
        moved = true;
      } else if (left_s > 0 && is - it < 2 && ready(&full[is % kStages], (is / kStages) & 1) &&
                 (!begins_s || ready(q_full, units & 1))) {
        // S of a tile whose keys have landed
        tc::fence_after();
        const uint64_t tile = dk + (static_cast<uint64_t>((is % kStages) * kTile) >> 4);
        const uint32_t to = tbase + kColS + (is & 1) * kTileKeys;
#pragma unroll
        for (int c = 0; c < kLatentRow / 16; ++c)
          tc::mma_ss(to, dq + (static_cast<uint64_t>((c / 4) * kSlab + (c % 4) * 32) >> 4),
                     tile + (static_cast<uint64_t>((c / 4) * 1024 + (c % 4) * 32) >> 4), id_s, c > 0);
        tc::commit(&bar_s[is & 1]);
        if (begins_s) ++units;
        begins_s = false;
        ++is;
        if (--left_s == 0) tc::commit(q_empty);
        moved = true;
      } else if (left_s == 0 && !end_s && ready(&job_full[job_s % kJobs], (job_s / kJobs) & 1)) {
        const Job& j = jobs[job_s % kJobs];
        end_s = j.rows == 0;
        left_s = end_s ? 0 : j.tile1 - j.tile0;
        begins_s = true;
        ++job_s;
        moved = true;
      }
      if (moved) {
        since = 0;
        idle = 0;
      } else if ((++idle & 255) == 0) {
        const unsigned long long t = globaltimer();
        if (since == 0) since = t;
        ok = __all_sync(0xffffffffu, t - since <= kWaitLimitNs) != 0;
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) raise_flag(a.flag, PKV_FLAG_TIMEOUT);
  } else {
    // ================= softmax, output =================
    const int g4 = lane >> 2, t4 = lane & 3, half = warp >> 2, w4 = warp & 3;
    const int ra = w4 * 16 + g4, rb = ra + 8;              // this thread's rows of the unit
    const uint32_t quarter = tbase + (static_cast<uint32_t>(w4 * 32) << 16);
    // its half of a row of P (rows ra and rb are in the 8-row groups 2 w4 and 2 w4 + 1)
    const uint32_t p_row = smem_u32(smem + kOffP) + 2 * w4 * 1024 + g4 * 128 + t4 * 4;
    const float sc = a.scale_log2;
    Unsplit begun{0, 0, 0};
    float* const ws_o = reinterpret_cast<float*>(wsp);
    float* const ws_lse = reinterpret_cast<float*>(wsp + ws.lse);
    // The warps meet at named barriers, which have no time limit: one whose wait gave up
    // goes on without waiting (its block is flagged, its rows unspecified).
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
    };
    // O has taken half h of tile t (the second half: all of it)
    auto wait_o = [&](uint32_t t, int h) {
      wait(&empty[(t % kStages) * 2 + h], (t / kStages) & 1);
    };
    for (uint32_t k = 0;; ++k) {
      if (tc::any_of(1, kSoftmax, !ok || !job_ready(k))) {
        ok = false;
        break;
      }
      const Job j = jobs[k % kJobs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&job_empty[k % kJobs]);
      if (j.rows == 0) break;
      const int64_t row0 = j.row0;
      const int rows = j.rows;
      const bool whole = j.first && j.last;
      const int slot = piece_slot(blockIdx.x, j.first != 0);
      if (j.pieces > 0) begun = Unsplit{row0, rows, j.pieces};
      if (j.tile0 >= j.tile1) {                            // (never a whole unit)
        if (threadIdx.x < rows) ws_lse[lse_at(threadIdx.x, slot, gridDim.x)] = kNoKeys;
        continue;
      }
      const bool valid_a = ra < rows, valid_b = rb < rows;
      auto limit = [&](int row) {
        return a.causal ? j.lead + static_cast<int>(static_cast<uint32_t>(j.first_row + row) /
                                                    static_cast<uint32_t>(a.hq))
                        : j.lead;
      };
      const int lim_a = limit(min(ra, rows - 1)), lim_b = limit(min(rb, rows - 1));
      const int lim_min = limit(0), kv_len = limit(rows - 1);
      bool spoilt = false;                                 // some rows see what others are spared
      float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
#pragma unroll 1
      for (int kt = j.tile0; kt < j.tile1; ++kt, ++it) {
        const int key0 = kt * kTileKeys;
        wait(&bar_s[it & 1], (it >> 1) & 1);
        tc::fence_after();
        uint32_t raw[16];
        tc::ld_tile16x32(quarter + kColS + (it & 1) * kTileKeys + half * 32, raw);
        tc::wait_ld(raw);
        float s[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __uint_as_float(raw[i]);
        // s[4 i + {0, 1}]: keys 8 i + 2 t4 + {0, 1} of row ra, s[4 i + {2, 3}] of row rb
        if (key0 + kTileKeys > lim_min) {
          // keys whose scores are non-finite in every row of the unit
          uint32_t b = 0xffffffffu;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool fin = (valid_a && isfinite(s[4 * (i / 2) + (i & 1)])) ||
                             (valid_b && isfinite(s[4 * (i / 2) + 2 + (i & 1)]));
            if (fin) b &= ~(1u << (8 * (i / 2) + 2 * t4 + (i & 1)));
          }
          tc::sync_named(1, kSoftmax);                     // (another tile's readers are done)
          if (threadIdx.x < 2) bad[threadIdx.x] = 0xffffffffu;
          tc::sync_named(1, kSoftmax);
          b = __reduce_and_sync(0xffffffffu, b);
          if (lane == 0) atomicAnd(&bad[half], b);
          tc::sync_named(1, kSoftmax);
          // 128 threads for each 32 keys, of the blocks that O takes; two rows at a time
          const int first = 32 * half;
          const int held = min(j.blocks * kBlock - key0, kTileKeys) - first;
          const int seen = kv_len - key0 - first;
          const int shown = lim_min - key0 - first;        // (to all rows)
          uint32_t zero = bad[half];
          if (shown > 0) zero &= shown < 32 ? ~0u << shown : 0u;
          if (seen < 32) zero &= seen <= 0 ? 0u : (1u << seen) - 1;
          spoilt |= zero != 0;
          if (seen < 32) zero |= seen <= 0 ? 0xffffffffu : ~0u << seen;
          if (held < 32) zero &= held <= 0 ? 0u : (1u << held) - 1;
          const int slab = threadIdx.x % 64 / 8, odd = threadIdx.x / 64 % 2;
          for (; zero != 0; zero &= zero - 1) {
            const int key = first + __ffs(zero) - 1;
            if ((key & 1) == odd)
              *reinterpret_cast<uint4*>(smem + kOffTiles + (it % kStages) * kTile +
                                        (key / 8) * kGroup + slab * 1024 + (key % 8) * 128 +
                                        (threadIdx.x % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int key = key0 + first + 8 * (i / 2) + 2 * t4 + (i & 1);
            float& x = s[4 * (i / 2) + (i & 1)];
            float& y = s[4 * (i / 2) + 2 + (i & 1)];
            x = key < lim_a ? x : -INFINITY;
            y = key < lim_b ? y : -INFINITY;
          }
        }
        float xa = fmaxf(s[0], s[1]), xb = fmaxf(s[2], s[3]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          xa = tc::max3(xa, s[4 * i], s[4 * i + 1]);
          xb = tc::max3(xb, s[4 * i + 2], s[4 * i + 3]);
        }
        // does any score exceed its row's reference by the slack?  (a piece's first tile
        // sets the references)
        const bool up = (valid_a && xa * sc > ma + kSlack) || (valid_b && xb * sc > mb + kSlack);
        if (tc::any_of(1, kSoftmax, up) || kt == j.tile0) {
          // the rows' maxima: over the four threads of a row, and both halves' warps
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, o));
            xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, o));
          }
          if (t4 == 0) {
            tops[half * kUnitRows + ra] = xa;
            tops[half * kUnitRows + rb] = xb;
          }
          tc::sync_named(1, kSoftmax);
          const float ca = fmaxf(ma, fmaxf(xa, tops[(half ^ 1) * kUnitRows + ra]) * sc);
          const float cb = fmaxf(mb, fmaxf(xb, tops[(half ^ 1) * kUnitRows + rb]) * sc);
          if (kt == j.tile0) {
            ma = ca;
            mb = cb;
          } else {
            const bool up_a = valid_a && ca > ma + kSlack, up_b = valid_b && cb > mb + kSlack;
            const float fa = up_a ? tc::exp2_fast(ma - ca) : 1.f;
            const float fb = up_b ? tc::exp2_fast(mb - cb) : 1.f;
            if (up_a) ma = ca;
            if (up_b) mb = cb;
            la *= fa;
            lb *= fb;
            if (t4 == 0 && half == 0) {
              factor[ra] = fa;
              factor[rb] = fb;
            }
            wait_o(it - 1, 1);
            tc::fence_after();
            tc::sync_named(1, kSoftmax);
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {                  // 32 rows of 128 dims at a time
              const uint32_t at = quarter + kColO + ((i & 2) + half) * kUnitRows + (i & 1) * 32;
              uint32_t v[32];
              tc::ld_row32(at, v);
              tc::wait_ld(v);
              const float4* f = reinterpret_cast<const float4*>(factor + (i & 1) * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 x = f[e];
                v[4 * e] = __float_as_uint(__uint_as_float(v[4 * e]) * x.x);
                v[4 * e + 1] = __float_as_uint(__uint_as_float(v[4 * e + 1]) * x.y);
                v[4 * e + 2] = __float_as_uint(__uint_as_float(v[4 * e + 2]) * x.z);
                v[4 * e + 3] = __float_as_uint(__uint_as_float(v[4 * e + 3]) * x.w);
              }
              tc::st_row32(at, v);
            }
            tc::wait_st();
            tc::fence_before();
          }
          // (either half's P lets the next product begin; the maxima are read)
          tc::sync_named(1, kSoftmax);
          tc::fence_after();
        }
        const float na = ma == -INFINITY ? 0.f : -ma, nb = mb == -INFINITY ? 0.f : -mb;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p0 = tc::exp2_fast(fmaf(s[4 * i], sc, na));
          const float p1 = tc::exp2_fast(fmaf(s[4 * i + 1], sc, na));
          const float p2 = tc::exp2_fast(fmaf(s[4 * i + 2], sc, nb));
          const float p3 = tc::exp2_fast(fmaf(s[4 * i + 3], sc, nb));
          la += p0 + p1;
          lb += p2 + p3;
          w[2 * i] = tc::pack_bf16(p0, p1);
          w[2 * i + 1] = tc::pack_bf16(p2, p3);
        }
        if (it > 0) wait_o(it - 1, half);                  // (it has read this half of P)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = p_row + (((i + 4 * half) ^ g4) << 4);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w[2 * i]) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(w[2 * i + 1]) : "memory");
        }
        tc::fence_async_smem();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[half]);
      }
      // ---- the piece's output ----
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, o);
        lb += __shfl_xor_sync(0xffffffffu, lb, o);
      }
      if (t4 == 0 && half == 1) {
        factor[ra] = la;
        factor[rb] = lb;
      }
      tc::sync_named(1, kSoftmax);
      if (t4 == 0 && half == 0) {
        la += factor[ra];
        lb += factor[rb];
        factor[ra] = la == 0.f ? 0.f : 1.f / la;
        factor[rb] = lb == 0.f ? 0.f : 1.f / lb;
        const float ea = la == 0.f ? -INFINITY : ma + tc::log2_fast(la);
        const float eb = lb == 0.f ? -INFINITY : mb + tc::log2_fast(lb);
        if (!whole) {
          if (valid_a) ws_lse[lse_at(ra, slot, gridDim.x)] = ea;
          if (valid_b) ws_lse[lse_at(rb, slot, gridDim.x)] = eb;
        } else if (a.lse_out != nullptr) {
          if (valid_a) a.lse_out[row0 + ra] = ea * kLn2;
          if (valid_b) a.lse_out[row0 + rb] = eb * kLn2;
        }
      }
      wait_o(it - 1, 1);
      tc::fence_after();
      spoilt = tc::any_of(1, kSoftmax, spoilt);
      // (lane = dim, column = row; 16 rows at a time)
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        const int first = (c & 3) * 16, tile = (c & 4) / 2 + half;
        const int dim = tile * 128 + w4 * 32 + lane;
        if (first >= rows) continue;
        uint32_t v[16];
        tc::ld_row16(quarter + kColO + tile * kUnitRows + first, v);
        float4 inv[4];                                     // (read before any store)
#pragma unroll
        for (int i = 0; i < 4; ++i) inv[i] = *reinterpret_cast<const float4*>(factor + first + 4 * i);
        tc::wait_ld(v);
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[4 * i] = __uint_as_float(v[4 * i]) * inv[i].x;
          f[4 * i + 1] = __uint_as_float(v[4 * i + 1]) * inv[i].y;
          f[4 * i + 2] = __uint_as_float(v[4 * i + 2]) * inv[i].z;
          f[4 * i + 3] = __uint_as_float(v[4 * i + 3]) * inv[i].w;
        }
        if (whole) {
          // two rows' pairs of dims: an even lane stores row i, its neighbour row i + 1
          __nv_bfloat16* to = a.out + (row0 + first + (lane & 1)) * kLatent + (dim & ~1);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? f[i] : f[i + 1], 1);
            if (first + i + (lane & 1) < rows)
              *reinterpret_cast<uint32_t*>(to + i * kLatent) =
                  (lane & 1) ? tc::pack_bf16(other, f[i + 1]) : tc::pack_bf16(f[i], other);
          }
        } else {
          float* to = ws_o + (static_cast<int64_t>(slot) * a.slot_rows + first) * kLatent + dim;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (first + i < rows) to[i * kLatent] = f[i];
        }
      }
      if (spoilt) {
        __syncwarp();                                      // (behind the warp's stores)
        const int32_t* table = a.block_table + static_cast<int64_t>(j.request) * a.max_blocks_per_seq;
        const int key0 = max(lim_min, j.tile0 * kTileKeys), key1 = min(kv_len, j.tile1 * kTileKeys);
        const int dim0 = half * 128 + w4 * 32 + lane;
        if (whole)
          spoil(a.out + row0 * kLatent, __ushort_as_bfloat16(0x7FFF), a.cache, table, a.num_blocks, a.hq,
                j.lead, j.first_row, rows, key0, key1, dim0);
        else
          spoil(ws_o + static_cast<int64_t>(slot) * a.slot_rows * kLatent, __int_as_float(0x7FC00000), a.cache,
                table, a.num_blocks, a.hq, j.lead, j.first_row, rows, key0, key1, dim0);
      }
      tc::fence_before();
      tc::sync_named(1, kSoftmax);                         // (the factors are free again)
    }
    if (threadIdx.x == 0) reinterpret_cast<Unsplit*>(wsp + ws.units)[blockIdx.x] = begun;
    if (!ok && lane == 0) raise_flag(a.flag, PKV_FLAG_TIMEOUT);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_free(tbase, kTmemCols);
}

// Merge of the units that one block of the first kernel begins and others end: with e_i a
// piece's log2 log-sum-exp and M their maximum, a row is sum 2^(e_i - M) o_i / sum 2^(e_i -
// M).  The rows of all such units are dealt out evenly over the grid.  A warp takes a quarter of
// a row's 512 elements: of all pieces of four rows, where these are at most four (a block then
// has eight rows), of two rows where they are at most eight, else of every eighth piece of one
// row, and the block's warps add up.  Lane i holds the weight of its warp's i-th piece;
// sixteen loads are in flight a thread, begun before the weights are there.  (Without the
// four-row form 64 requests take 45.0 us instead of 43.0: twice as many rounds.)
struct Merge {
  const float *o, *lse;
  int slot_rows, blocks, first;                  // the block that begins the unit
  // where piece p of a row lies
  __device__ __forceinline__ int slot(int p) const { return piece_slot(first + p, p == 0); }
  __device__ __forceinline__ float log_sum(int row, int p) const {
    return __ldcg(lse + lse_at(row, slot(p), blocks));
  }
  __device__ __forceinline__ float4 values(int row, int p, int column) const {
    const int64_t at = static_cast<int64_t>(slot(p)) * slot_rows + row;
    return __ldcg(reinterpret_cast<const float4*>(o + at * kLatent) + column);
  }
};

// The lanes' weights within each run of `Lanes` (a piece without keys, weight -1 here, holds
// no rows: whatever lies there is left out), their maximum and their sum.  A piece whose keys
// all weigh nothing has weight 0: its rows are 0, or the NaN that 0 times an infinity is.
template <int Lanes>
__device__ __forceinline__ void weigh(float e, float& m, float& w, float& total) {
  const bool none = e == kNoKeys;
  m = none ? -INFINITY : e;
#pragma unroll
  for (int k = 1; k < Lanes; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  w = none ? -1.f : e == -INFINITY ? 0.f : tc::exp2_fast(e - m);
  total = w < 0.f ? 0.f : w;
#pragma unroll
  for (int k = 1; k < Lanes; k <<= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
}

__device__ __forceinline__ void weighted(float4& y, float w, const float4& x) {
  y.x = w < 0.f ? y.x : fmaf(w, x.x, y.x);
  y.y = w < 0.f ? y.y : fmaf(w, x.y, y.y);
  y.z = w < 0.f ? y.z : fmaf(w, x.z, y.z);
  y.w = w < 0.f ? y.w : fmaf(w, x.w, y.w);
}

// One warp: its quarter of kMergeBatch / Span rows from `row` on, of at most Span pieces.
template <int Span>
__device__ __forceinline__ void merge_few(const LatentArgs& a, const Merge& at, const Unsplit& u,
                                          int row, int quarter, int lane) {
  constexpr int kRows = kMergeBatch / Span;
  const int column = quarter * 32 + lane;
  const bool mine = lane < kMergeBatch && lane % Span < u.pieces && row + lane / Span < u.rows;
  const float e = mine ? at.log_sum(row + lane / Span, lane % Span) : kNoKeys;
  float4 x[kMergeBatch];
#pragma unroll
  for (int k = 0; k < kMergeBatch; ++k) {
    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k % Span < u.pieces && row + k / Span < u.rows)
      x[k] = at.values(row + k / Span, k % Span, column);
  }
  float m, w, total;
  weigh<Span>(e, m, w, total);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < Span; ++k)
      weighted(y, __shfl_sync(0xffffffffu, w, r * Span + k), x[r * Span + k]);
    const float sum = __shfl_sync(0xffffffffu, total, r * Span);
    const float top = __shfl_sync(0xffffffffu, m, r * Span);
    if (row + r >= u.rows) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    reinterpret_cast<uint2*>(a.out + (u.row + row + r) * kLatent)[column] =
        make_uint2(tc::pack_bf16(y.x * inv, y.y * inv), tc::pack_bf16(y.z * inv, y.w * inv));
    if (column == 0 && a.lse_out != nullptr)
      a.lse_out[u.row + row + r] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

__global__ void __launch_bounds__(kMergeThreads, 2)
    latent_merge_kernel(const LatentArgs a, int blocks) {
  extern __shared__ int4 units_raw[];            // [blocks], then [blocks + 1]: items before each
  Unsplit* units = reinterpret_cast<Unsplit*>(units_raw);
  int* upto = reinterpret_cast<int*>(units + blocks);
  __shared__ float4 part[kMergeWarps][32];
  __shared__ float2 stat[kMergeWarps];           // a warp's maximum and sum
  __shared__ int sums[kMergeWarps];
  pdl_launch_dependents();
  pdl_wait_primary();
  const Layout ws = layout(blocks);
  const uint8_t* wsp = static_cast<const uint8_t*>(a.workspace);
  Merge at{reinterpret_cast<const float*>(wsp), reinterpret_cast<const float*>(wsp + ws.lse),
           a.slot_rows, blocks, 0};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  {
    // (no more blocks than threads)
    int items = 0;
    if (threadIdx.x < blocks) {
      const Unsplit u = reinterpret_cast<const Unsplit*>(wsp + ws.units)[threadIdx.x];
      units[threadIdx.x] = u;
      items = u.pieces == 0 ? 0
              : u.pieces > 8 ? 4 * u.rows
              : u.pieces > 4 ? (u.rows + 3) / 4 : (u.rows + 7) / 8;
    }
    int sum = items;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += y;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k)
      if (k < warp) sum += sums[k];
    if (threadIdx.x < blocks) upto[threadIdx.x + 1] = sum;
    if (threadIdx.x == 0) upto[0] = 0;
    __syncthreads();
  }
  for (int item = blockIdx.x; item < upto[blocks]; item += gridDim.x) {
    int lo = 0;                                  // upto[lo] <= item < upto[lo + 1]
#pragma unroll
    for (int k = 0; k < kMergeWarps; ++k) {
      const int c = k * 32 + lane;
      lo += __popc(__ballot_sync(0xffffffffu, c < blocks && upto[c + 1] <= item));
    }
    const Unsplit u = units[lo];
    const int nth = item - upto[lo];
    at.first = lo;
    if (u.pieces <= 4) {
      merge_few<4>(a, at, u, nth * 8 + warp / 4 * 4, warp % 4, lane);
      continue;
    }
    if (u.pieces <= 8) {
      merge_few<8>(a, at, u, nth * 4 + warp / 4 * 2, warp % 4, lane);
      continue;
    }
    const int row = nth / 4, quarter = nth % 4;
    auto piece_of = [&](int i) { return warp + i * kMergeWarps; };   // (32 at most a warp)
    const float e = piece_of(lane) < u.pieces ? at.log_sum(row, piece_of(lane)) : kNoKeys;
    float4 x[kMergeBatch], acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m, w, total;
#pragma unroll 1
    for (int i0 = 0; i0 == 0 || piece_of(i0) < u.pieces; i0 += kMergeBatch) {
#pragma unroll
      for (int k = 0; k < kMergeBatch; ++k) {
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (piece_of(i0 + k) < u.pieces) x[k] = at.values(row, piece_of(i0 + k), quarter * 32 + lane);
      }
      if (i0 == 0) weigh<32>(e, m, w, total);
#pragma unroll
      for (int k = 0; k < kMergeBatch; ++k) weighted(acc, __shfl_sync(0xffffffffu, w, i0 + k), x[k]);
    }
    part[warp][lane] = acc;
    if (lane == 0) stat[warp] = make_float2(m, total);
    __syncthreads();
    if (threadIdx.x < 64) {
      m = stat[0].x;
#pragma unroll
      for (int k = 1; k < kMergeWarps; ++k) m = fmaxf(m, stat[k].x);
      float2 y = make_float2(0.f, 0.f);
      total = 0.f;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) {
        const float2 z = reinterpret_cast<const float2*>(part[k])[threadIdx.x];
        const float f = stat[k].x == -INFINITY ? 0.f : tc::exp2_fast(stat[k].x - m);
        y.x = fmaf(f, z.x, y.x);
        y.y = fmaf(f, z.y, y.y);
        total = fmaf(f, stat[k].y, total);
      }
      const float inv = total == 0.f ? 0.f : 1.f / total;
      reinterpret_cast<uint32_t*>(a.out + (u.row + row) * kLatent)[quarter * 64 + threadIdx.x] =
          tc::pack_bf16(y.x * inv, y.y * inv);
      if (threadIdx.x == 0 && quarter == 0 && a.lse_out != nullptr)
        a.lse_out[u.row + row] = total == 0.f ? -INFINITY : (m + log2f(total)) * kLn2;
    }
    __syncthreads();
  }
}

cudaError_t launch_latent(LatentArgs a, const CUtensorMap& qmap, const CUtensorMap& cmap,
                          int num_sms, cudaStream_t stream) {
  const int blocks = std::min(num_sms, kMostBlocks);
  // (few rows: their partials lie close together, on few pages of memory)
  a.slot_rows = static_cast<int>(
      std::min<int64_t>(kUnitRows, static_cast<int64_t>(a.max_query_len) * a.hq));
  static DeviceSet done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!done.has(dev)) {
    e = cudaFuncSetAttribute(latent_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.add(dev);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_kernel, qmap, cmap, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(2 * blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = blocks * sizeof(Unsplit) + (blocks + 1) * sizeof(int);
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel, a, blocks);
}

size_t latent_workspace_bytes(int num_sms) {
  return layout(std::min(num_sms, kMostBlocks)).bytes;
}

}  // namespace pkv
