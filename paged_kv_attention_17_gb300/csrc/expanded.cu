// Latent attention in the expanded form, on the 5th-generation tensor cores (tcgen05 +
// TMEM + TMA): keys of 128 + 64 elements, the last 64 shared by the heads, values of 128,
// contiguous rows.
//
// "Inside the engine: kernels, CUDA graphs and the life of a request", sections "Never
// materialise the TxT matrix" (a block of queries stays on chip while K/V tiles stream past
// it) and "Prefill has a full grid ..." (a tile per block of queries, keys not split).
//
// One block = 256 query rows of one request and head, as two tiles of 128; a key tile is
// 128 keys, which feeds both.  Where that would leave SMs idle a block is one tile, whose
// key tiles the two warpgroups take in turn (below: t is then the warpgroup, V(k) its next
// tile), and their two results are added up.
//   warps 0-3 and 4-7: one softmax warpgroup per query tile, one row per thread: the S row
//     is read from TMEM, masked only on tiles that cross a row's limit, exponentiated in the
//     log2 domain and written back into TMEM as bf16 P over its own S;
//   warp 8 loads K (64-column slabs through a ring of four, so that the next tile's first
//     slab is there before this one's last is done), warp 9 the queries and V (two stages);
//   warp 11 cleans V where rows of the block do not see all of a tile's keys (below);
//   warp 10 issues the MMAs in the order P0 V(k), S0(k + 1), P1 V(k), S1(k + 1): one tile's
//     softmax runs beside the other's products.
// Shared memory: 96 KB of queries, 64 KB of K, 64 KB of V.  A key tile is 2560 cycles of
// MMAs for both query tiles (12 of 192 / 16 steps and 8 of 128 / 16, 64 cycles each) and 2048
// of exponentials; it takes about 3500, which is a tile's chain from scores through softmax and
// P V to the next scores: P lies over its own S, as TMEM has no room beside two S and two O.
// Measured: 8192 tokens of 32 heads, causal, in 500 us (498 to 514 from card to card), 1.37
// PFLOP/s (72% of a library matrix product's rate; the tensor pipe is busy for 62% of the time, with
// the units' starts, their ends and the tiles that the causal limit crosses); five prompts of 130
// to 777 tokens on up to 333 cached, 12 heads, 23 us.
// Tried and slower: P handed on in two halves (519 us for the 8192 tokens: the second wait and
// store cost the softmax warps more than the earlier product gives), an eighth or a quarter
// of the exponentials as polynomials on the FMA units (517, 561 us: the warps' instructions
// bound them, not the exponential unit).
//
// The running maximum is a reference that moves only when a row's maximum is 8 log2 units
// above it (p <= 2^8; O is rescaled rarely).  In the tiles that cross a row's limit, V rows
// behind the block's last key are zeroed, and so are the infinities and NaN in the rows that
// some of the block's rows do not see (0 times them would be a NaN); the rows that do see
// them take them at the end.
#include <algorithm>

#include "device_set.h"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 384;
constexpr int kRows = 128;                       // rows of a query tile
constexpr int kKeys = 128;
constexpr int kSlab = 128 * 128;                 // 128 rows of 64 bf16
constexpr int kQSlabs = kExpandedRow / 64;       // 3, as many as of K
constexpr int kKSlots = 4, kVStages = 2;
constexpr int kLoadK = 8, kLoadV = 9, kMmaWarp = 10, kCleanWarp = 11;
constexpr int kOffK = 2 * kQSlabs * kSlab;
constexpr int kOffV = kOffK + kKSlots * kSlab;
constexpr int kOffBars = kOffV + kVStages * 2 * kSlab;
// q, k_full[], k_empty[], v_full[], v_empty[], v_clean[], s[2], p[2], o[2]
constexpr int kBars = 1 + 2 * kKSlots + 3 * kVStages + 6;
constexpr int kOffMisc = (kOffBars + kBars * 8 + 15) / 16 * 16;   // unit[2], tmem, any, first[3][128]
constexpr int kSmem = kOffMisc + 16 + 3 * kNope * 4 + 1024;
static_assert(kSmem <= 232448, "shared memory of the expanded kernel");
constexpr int kTmemCols = 512;
constexpr int kColO = 2 * kKeys;                 // S_t at 128 t, O_t at 256 + 128 t
constexpr float kSlack = 8.f;
constexpr int kFewUnits = 1;                     // blocks of two tiles an SM

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0;
}
// The magnitudes' bits of two bf16, the larger of these and of `m` each.
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7FFF7FFFu);
}

// The infinities and NaN that a row sees, of those that V was cleaned of.
__device__ __forceinline__ void with_seen(float (&f)[32], const int* first, int lim) {
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    if (first[e] < lim) f[e] += INFINITY;
    if (first[kNope + e] < lim) f[e] -= INFINITY;
    if (first[2 * kNope + e] < lim) f[e] = __int_as_float(0x7FC00000);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(tc::pack_bf16(f[0], f[1]), tc::pack_bf16(f[2], f[3]), tc::pack_bf16(f[4], f[5]),
                    tc::pack_bf16(f[6], f[7]));
}

}  // namespace

// A block's rows are two tiles of 128; or with Halves one, whose key tiles the two softmax
// warpgroups take in turn and whose two sums are added up at the end.
template <bool Halves>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap qmap,
                    const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap rmap,
                    const __grid_constant__ CUtensorMap vmap, const ExpandedArgs a) {
  constexpr int kUnit = Halves ? kRows : 2 * kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bar_q = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* k_full = bar_q + 1;
  uint64_t* k_empty = k_full + kKSlots;
  uint64_t* v_full = k_empty + kKSlots;
  uint64_t* v_empty = v_full + kVStages;
  uint64_t* v_clean = v_empty + kVStages;
  uint64_t* bar_s = v_clean + kVStages;          // [tile]
  uint64_t* bar_p = bar_s + 2;
  uint64_t* bar_o = bar_s + 4;
  int* misc = reinterpret_cast<int*>(smem + kOffMisc);   // request, unit, tmem, any non-finite
  // [+inf, -inf, NaN][dim]: the first key that has it there, of those that not all rows see
  int* first = misc + 4;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // heads vary fastest, the requests' last (heaviest) units come first
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.hq));
  const int nth = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.hq));
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (uint64_t* b = bar_q; b < bar_q + kBars; ++b)
      mbar_init(b, b >= bar_p && b < bar_o ? 4 : 1);     // (P: a lane of each warp)
    fence_mbar_init();
    misc[3] = 0;
  }
  for (int e = threadIdx.x; e < 3 * kNope; e += kThreads) first[e] = 0x7FFFFFFF;
  pdl_wait_primary();
  // ---- which unit: warp 0 adds up the requests' units, four requests a lane where there are
  // many (1000 of 16 tokens, 8 heads: 600 us, one by one 803; 256 of 64, 16 heads: 235 and 286) ----
  if (warp == 0) {
    const int each = a.num_seqs <= 32 ? 1 : 4;
    int64_t base = 0;
    bool found = false;
    if (lane == 0) misc[0] = -1;
    __syncwarp();
    // (block 0 looks at every request: it tells of the invalid ones)
    for (int r0 = 0; r0 < a.num_seqs && (!found || blockIdx.x == 0); r0 += 32 * each) {
      int units[4], sum = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + lane * each + k;
        units[k] = 0;
        if (k < each && r < a.num_seqs) {
          const int q0 = __ldg(a.qsl + r), q1 = __ldg(a.qsl + r + 1);
          const int k0 = __ldg(a.ksl + r), k1 = __ldg(a.ksl + r + 1);
          const int64_t n = static_cast<int64_t>(q1) - q0, m = static_cast<int64_t>(k1) - k0;
          const bool valid = q0 >= 0 && n >= 0 && q1 <= a.num_tokens && n <= a.max_query_len &&
                             k0 >= 0 && m >= 0 && k1 <= a.num_keys && m <= a.max_key_len;
          if (blockIdx.x == 0 && (!valid || (r == 0 && (q0 != 0 || k0 != 0))))
            raise_flag(a.flag, PKV_FLAG_BAD_LENGTHS);
          units[k] = valid ? static_cast<int>((n + kUnit - 1) / kUnit) : 0;
        }
        sum += units[k];
      }
      int64_t upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const int64_t total = __shfl_sync(0xffffffffu, upto, 31);
      if (!found && nth < base + total) {
        found = true;
        int64_t before = base + upto - sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (nth >= before && nth < before + units[k]) {
            misc[0] = r0 + lane * each + k;
            misc[1] = units[k] - 1 - static_cast<int>(nth - before);
          }
          before += units[k];
        }
      }
      base += total;
    }
  }
  __syncthreads();
  const int r = misc[0];
  if (r < 0) return;                             // past the last unit
  const int i0 = misc[1] * kUnit;                // the unit's first row of the request
  const int q0 = __ldg(a.qsl + r), n = __ldg(a.qsl + r + 1) - q0;
  const int k0 = __ldg(a.ksl + r), m = __ldg(a.ksl + r + 1) - k0;
  // keys that row i sees, and key tiles of the two warpgroups (none without rows)
  auto limit = [&](int i) { return a.causal ? min(max(m - n + i + 1, 0), m) : m; };
  const int rows = min(kUnit, n - i0);
  const int kv_len = limit(i0 + rows - 1), lim_min = limit(i0);
  const int all = (kv_len + kKeys - 1) / kKeys;
  const int ntk0 = Halves ? (all + 1) / 2 : (limit(i0 + min(rows, kRows) - 1) + kKeys - 1) / kKeys;
  const int ntk1 = Halves ? all / 2 : rows > kRows ? all : 0;
  const int ntk = Halves ? all : max(ntk0, ntk1);
  if (ntk == 0) {                                // no row sees a key
    for (int i = threadIdx.x; i < rows * (kNope / 8); i += kThreads) {
      const int64_t row = static_cast<int64_t>(q0 + i0 + i / (kNope / 8)) * a.hq + h;
      reinterpret_cast<uint4*>(a.out + row * kNope)[i % (kNope / 8)] = make_uint4(0, 0, 0, 0);
      if (a.lse_out != nullptr && i % (kNope / 8) == 0) a.lse_out[row] = -INFINITY;
    }
    return;
  }
  // tiles from this one on hold keys that some row of the block does not see
  const int kt_edge = lim_min / kKeys;
  if (warp == kMmaWarp) tc::tmem_alloc(&misc[2], kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = static_cast<uint32_t>(misc[2]);
  bool ok = true;

  if (warp == kLoadK) {
    // ================= K: slab 3 kt + j through slot (3 kt + j) % 4 =================
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_last();
      int s = 0;
      for (; s < 3 * ntk; ++s) {
        const int slot = s % kKSlots, j = s % 3, key = k0 + s / 3 * kKeys;
        if (s >= kKSlots && !(ok = mbar_wait(&k_empty[slot], ((s / kKSlots) - 1) & 1))) break;
        uint8_t* to = smem + kOffK + slot * kSlab;
        mbar_arrive_expect_tx(&k_full[slot], kSlab);
        if (j < 2) tma_load_3d(to, &kmap, &k_full[slot], j * 64, h, key, policy);
        else tc::load_2d(to, &rmap, &k_full[slot], 0, key, policy);
      }
      if (!ok) {
        raise_flag(a.flag, PKV_FLAG_TIMEOUT);
        for (int x = max(0, s - kKSlots); x < s; ++x)
          mbar_wait(&k_full[x % kKSlots], (x / kKSlots) & 1);
      }
    }
  } else if (warp == kLoadV) {
    // ================= queries, V =================
    if (lane == 0) {
      const uint64_t policy = l2_policy_evict_last(), once = l2_policy_evict_first();
      const int tiles = rows > kRows ? 2 : 1;
      mbar_arrive_expect_tx(bar_q, tiles * kQSlabs * kSlab);
      for (int t = 0; t < tiles; ++t)
        for (int j = 0; j < kQSlabs; ++j)
          tma_load_3d(smem + (t * kQSlabs + j) * kSlab, &qmap, bar_q, j * 64, h,
                      q0 + i0 + t * kRows, once);
      int kt = 0;
      for (; kt < ntk; ++kt) {
        const int st = kt % kVStages;
        if (kt >= kVStages && !(ok = mbar_wait(&v_empty[st], ((kt / kVStages) - 1) & 1))) break;
        uint8_t* to = smem + kOffV + st * 2 * kSlab;
        mbar_arrive_expect_tx(&v_full[st], 2 * kSlab);
        tma_load_3d(to, &vmap, &v_full[st], 0, h, k0 + kt * kKeys, policy);
        tma_load_3d(to + kSlab, &vmap, &v_full[st], 64, h, k0 + kt * kKeys, policy);
      }
      if (!ok) {
        raise_flag(a.flag, PKV_FLAG_TIMEOUT);
        for (int x = max(0, kt - kVStages); x < kt; ++x)
          mbar_wait(&v_full[x % kVStages], (x / kVStages) & 1);
      }
      mbar_wait(bar_q, 0);
    }
  } else if (warp == kMmaWarp) {
    // ================= MMAs (the whole warp: see mma_ss) =================
    constexpr uint32_t id_s = tc::instr_desc(kRows, kKeys, false, false);
    constexpr uint32_t id_o = tc::instr_desc(kRows, kNope, false, true);
    const uint64_t dq = tc::smem_desc(smem_u32(smem), 16, 1024);
    const uint64_t dk = tc::smem_desc(smem_u32(smem + kOffK), 16, 1024);
    const uint64_t dv = tc::smem_desc(smem_u32(smem + kOffV), kSlab, 1024);
    // S_t of key tile kt, slab by slab as they land; `last`: no other tile will use them
    auto scores = [&](int t, int kt, bool last) {
#pragma unroll
      for (int j = 0; j < kQSlabs; ++j) {
        const int s = 3 * kt + j, slot = s % kKSlots;
        if (!(ok = ok && wait_all(&k_full[slot], (s / kKSlots) & 1))) return;
        tc::fence_after();
        const uint64_t qa = dq + (static_cast<uint64_t>(((Halves ? 0 : t * kQSlabs) + j) * kSlab) >> 4);
        const uint64_t kb = dk + (static_cast<uint64_t>(slot * kSlab) >> 4);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tc::mma_ss(tbase + t * kKeys, qa + c * 2, kb + c * 2, id_s, j > 0 || c > 0);
        if (last) tc::commit(&k_empty[slot]);
      }
      tc::commit(&bar_s[t]);
    };
    // O_t += P_t V of key tile kt, its nth, 16 keys a step
    auto values = [&](int t, int kt, int nth, bool end) {
      if (!(ok = ok && wait_all(&bar_p[t], nth & 1))) return;
      tc::fence_after();
      const uint64_t vb = dv + (static_cast<uint64_t>(kt % kVStages * 2 * kSlab) >> 4);
#pragma unroll
      for (int c = 0; c < kKeys / 16; ++c)
        tc::mma_ts(tbase + kColO + t * kNope, tbase + t * kKeys + c * 8,
                   vb + (static_cast<uint64_t>(c * 2048) >> 4), id_o, nth > 0 || c > 0);
      if (end) tc::commit(&bar_o[t]);
    };
    ok = wait_all(bar_q, 0);
    if constexpr (Halves) {
      scores(0, 0, true);
      if (ntk > 1) scores(1, 1, true);
      auto step = [&](int t, int kt) {
        if (kt >= ntk || !(ok = ok && wait_all(&v_clean[t], (kt / 2) & 1))) return;
        tc::fence_after();
        values(t, kt, kt / 2, kt + 2 >= ntk);
        tc::commit(&v_empty[t]);
        if (kt + 2 < ntk) scores(t, kt + 2, true);
      };
      for (int kt = 0; ok && kt < ntk; kt += 2) {
        step(0, kt);
        step(1, kt + 1);
      }
    } else {
      if (ntk0 > 0) scores(0, 0, ntk1 == 0);
      if (ntk1 > 0) scores(1, 0, true);
      for (int kt = 0; ok && kt < ntk; ++kt) {
        if (!(ok = wait_all(&v_clean[kt % kVStages], (kt / kVStages) & 1))) break;
        tc::fence_after();
        if (kt < ntk0) values(0, kt, kt, kt + 1 == ntk0);
        if (kt + 1 < ntk0) scores(0, kt + 1, kt + 1 >= ntk1);
        if (kt < ntk1) values(1, kt, kt, kt + 1 == ntk1);
        tc::commit(&v_empty[kt % kVStages]);
        if (kt + 1 < ntk1) scores(1, kt + 1, true);
      }
    }
    if (!ok && lane == 0) raise_flag(a.flag, PKV_FLAG_TIMEOUT);
  } else if (warp == kCleanWarp) {
    // ================= V rows that some row of the block does not see =================
    // (it hands on every tile, so that it never falls behind the barriers' phases)
    for (int kt = 0; ok && kt < ntk; ++kt) {
      const int st = kt % kVStages;
      if (!(ok = wait_all(&v_full[st], (kt / kVStages) & 1))) break;
#pragma unroll 1
      for (int row = kt < kt_edge ? kKeys : lane; row < kKeys; row += 32) {
        const int key = kt * kKeys + row;
        if (key < lim_min) continue;
        uint8_t* vrow = smem + kOffV + st * 2 * kSlab + row * 128;
        if (key >= kv_len) {                             // behind the last key
#pragma unroll
          for (int c = 0; c < 16; ++c)
            *reinterpret_cast<uint4*>(vrow + (c / 8) * kSlab + c % 8 * 16) = make_uint4(0, 0, 0, 0);
          continue;
        }
        uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 w = *reinterpret_cast<const uint4*>(vrow + (c / 8) * kSlab + ((c ^ row) & 7) * 16);
          top[0] = larger(top[0], w.x);
          top[1] = larger(top[1], w.y);
          top[2] = larger(top[2], w.z);
          top[3] = larger(top[3], w.w);
        }
        const uint32_t m = larger(larger(top[0], top[1]), larger(top[2], top[3]));
        if ((m & 0xFFFFu) < 0x7F80u && m < 0x7F800000u) continue;   // no infinity, no NaN
#pragma unroll 1
        for (int e = 0; e < kNope; ++e) {
          uint16_t* x = reinterpret_cast<uint16_t*>(vrow + (e / 64) * kSlab +
                                                    (((e / 8) ^ row) & 7) * 16 + e % 8 * 2);
          if ((*x & 0x7F80u) != 0x7F80u) continue;
          const int kind = (*x & 0x7Fu) != 0 ? 2 : *x >> 15;
          *x = 0;
          atomicMin(&first[kind * kNope + e], key);
          misc[3] = 1;
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_clean[st]);
    }
    if (!ok && lane == 0) raise_flag(a.flag, PKV_FLAG_TIMEOUT);
  } else {
    // ================= softmax, output: thread = row of tile t =================
    const int t = warp >> 2, row = threadIdx.x & (kRows - 1);
    const int tiles = t == 0 ? ntk0 : ntk1;
    const int own = Halves ? 0 : t * kRows;              // the tile's first row of the unit
    const int i = i0 + own + row;
    const bool real = own + row < rows;
    const int lim = limit(min(i, n - 1));                // padding rows mirror the last
    const int t_min = limit(min(i0 + own, n - 1));    // smallest of the tile
    const uint32_t lane_base = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = lane_base + t * kKeys, t_o = lane_base + kColO + t * kNope;
    const float sc = a.scale_log2;
    float mr = -INFINITY, l = 0.f;
    for (int kt = 0; ok && kt < tiles; ++kt) {
      const int key0 = (Halves ? 2 * kt + t : kt) * kKeys;
      if (!(ok = wait_all(&bar_s[t], kt & 1))) break;
      tc::fence_after();
      float s[kKeys];
      {
        uint32_t x0[32], x1[32], x2[32], x3[32];         // all four loads in flight
        tc::ld_row32(t_s, x0);
        tc::ld_row32(t_s + 32, x1);
        tc::ld_row32(t_s + 64, x2);
        tc::ld_row32(t_s + 96, x3);
        tc::wait_ld(x0);
        tc::wait_ld(x1);
        tc::wait_ld(x2);
        tc::wait_ld(x3);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s[c] = __uint_as_float(x0[c]);
          s[32 + c] = __uint_as_float(x1[c]);
          s[64 + c] = __uint_as_float(x2[c]);
          s[96 + c] = __uint_as_float(x3[c]);
        }
      }
      if (key0 + kKeys > t_min) {                        // a tile crossing a row's limit
#pragma unroll
        for (int c = 0; c < kKeys; ++c) s[c] = key0 + c < lim ? s[c] : -INFINITY;
      }
      float mx[8];                                       // 8 independent chains
#pragma unroll
      for (int j = 0; j < 8; ++j) mx[j] = fmaxf(s[j], s[j + 8]);
#pragma unroll
      for (int c = 16; c < kKeys; c += 16)
#pragma unroll
        for (int j = 0; j < 8; ++j) mx[j] = tc::max3(mx[j], s[c + j], s[c + 8 + j]);
      const float top = tc::max3(tc::max3(mx[0], mx[1], mx[2]), tc::max3(mx[3], mx[4], mx[5]),
                                 fmaxf(mx[6], mx[7]));
      const float cand = fmaxf(mr, top * sc);
      const float mn = cand > mr + kSlack ? cand : mr;
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = tc::exp2_fast(mr - ref);
      const tc::Pair sc2 = tc::pair(sc, sc), ref2 = tc::pair(-ref, -ref);
      tc::Pair sum4[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < kKeys / 2; ++j) {
        const float2 x = tc::unpair(tc::fma2(tc::pair(s[2 * j], s[2 * j + 1]), sc2, ref2));
        s[2 * j] = tc::exp2_fast(x.x);
        s[2 * j + 1] = tc::exp2_fast(x.y);
        sum4[j & 3] = tc::add2(sum4[j & 3], tc::pair(s[2 * j], s[2 * j + 1]));
      }
      const float2 sum = tc::unpair(tc::add2(tc::add2(sum4[0], sum4[1]), tc::add2(sum4[2], sum4[3])));
      l = l * alpha + (sum.x + sum.y);
      mr = mn;
      // P over the first 64 columns of this row's S, whose scores are read
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = tc::pack_bf16(s[64 * c + 2 * j], s[64 * c + 2 * j + 1]);
        tc::st_row32(t_s + 32 * c, w);
      }
      // (the previous P.V of this tile is done: it was issued before these scores)
      if (kt > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < kNope / 32; ++c) {
          uint32_t v[32];
          tc::ld_row32(t_o + c * 32, v);
          tc::wait_ld(v);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
          tc::st_row32(t_o + c * 32, v);
        }
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_p[t]);
    }
    if constexpr (Halves) {
      // ---- the halves of a row: m = max m_t, O = sum 2^(m_t - m) O_t / sum 2^(m_t - m) l_t ----
      // Each thread finishes half of its row's elements and hands the other half over
      // through shared memory, where the keys were ([chunk of 4][row]); the rows go out as below.
      if (ok && tiles > 0) ok = wait_all(&bar_o[t], 0);
      tc::fence_after();
      tc::sync_named(1, 2 * kRows);                      // (no product reads shared memory any more)
      float4* const over = reinterpret_cast<float4*>(smem + kOffK) + row;
      float2* const stats = reinterpret_cast<float2*>(smem + kOffV) + row;
      stats[t * kRows] = make_float2(mr, l);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tc::ld_row32(t_o + (1 - t) * (kNope / 2) + c * 32, v);
        tc::wait_ld(v);
#pragma unroll
        for (int e = 0; e < 8; ++e)                      // (without tiles TMEM holds nothing yet)
          over[(t * 16 + c * 8 + e) * kRows] =
              tiles == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                         : make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                       __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
      }
      tc::sync_named(1, 2 * kRows);
      const float2 other = stats[(1 - t) * kRows];
      const float m2 = fmaxf(mr, other.x);
      const float mine = mr == -INFINITY ? 0.f : tc::exp2_fast(mr - m2);
      const float its = other.x == -INFINITY ? 0.f : tc::exp2_fast(other.x - m2);
      const float sum = l * mine + other.y * its;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const bool any = *reinterpret_cast<volatile int*>(&misc[3]) != 0;
      uint8_t* const stage = smem + t * kSlab + (warp & 3) * (32 * kNope);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
        tc::ld_row32(t_o + t * (kNope / 2) + c * 32, v);
        tc::wait_ld(v);
        float f[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 x = over[((1 - t) * 16 + c * 8 + e) * kRows];
          const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            f[4 * e + k] = ((tiles == 0 ? 0.f : __uint_as_float(v[4 * e + k]) * mine) + y[k] * its) * inv;
        }
        if (any) with_seen(f, first + t * (kNope / 2) + c * 32, lim);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(stage + lane * kNope + ((c * 4 + e) ^ (lane & 7)) * 16) = pack8(f + 8 * e);
      }
      __syncwarp();
      const int row0 = (warp & 3) * 32, chunk = lane & 7;
      __nv_bfloat16* to = a.out + (static_cast<int64_t>(q0 + i0 + row0) * a.hq + h) * kNope +
                          t * (kNope / 2) + chunk * 8;
#pragma unroll 4
      for (int e = lane >> 3; e < 32; e += 4) {
        if (!ok || row0 + e >= rows) break;
        *reinterpret_cast<uint4*>(to + static_cast<int64_t>(e) * a.hq * kNope) =
            *reinterpret_cast<const uint4*>(stage + e * kNope + (chunk ^ (e & 7)) * 16);
      }
      if (ok && real && t == 0 && a.lse_out != nullptr)
        a.lse_out[static_cast<int64_t>(q0 + i) * a.hq + h] =
            sum == 0.f ? -INFINITY : (m2 + tc::log2_fast(sum)) * kLn2;
    } else if (ok && tiles > 0 && (ok = wait_all(&bar_o[t], 0))) {
      // ---- O row / l ----
      tc::fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool any = *reinterpret_cast<volatile int*>(&misc[3]) != 0;
      // The rows go out through shared memory, where this tile's queries were (its scores are
      // all done): a thread has a row, but a warp stores two whole rows at a time.  Chunk c
      // (16 bytes) of row r lies at place c ^ (r % 16): no bank conflicts either way.
      uint8_t* const stage = smem + t * kQSlabs * kSlab + (warp & 3) * (32 * kNope * 2);
#pragma unroll 1
      for (int c = 0; c < kNope / 32; ++c) {
        uint32_t v[32];
        tc::ld_row32(t_o + c * 32, v);
        tc::wait_ld(v);
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]) * inv;
        if (any) with_seen(f, first + c * 32, lim);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4*>(stage + lane * (kNope * 2) + ((c * 4 + e) ^ (lane & 15)) * 16) =
              pack8(f + 8 * e);
      }
      __syncwarp();
      const int row0 = t * kRows + (warp & 3) * 32, chunk = lane & 15;
      __nv_bfloat16* to = a.out + (static_cast<int64_t>(q0 + i0 + row0) * a.hq + h) * kNope + chunk * 8;
#pragma unroll 4
      for (int e = lane >> 4; e < 32; e += 2) {
        if (row0 + e >= rows) break;
        *reinterpret_cast<uint4*>(to + static_cast<int64_t>(e) * a.hq * kNope) =
            *reinterpret_cast<const uint4*>(stage + e * (kNope * 2) + (chunk ^ (e & 15)) * 16);
      }
      if (real && a.lse_out != nullptr)
        a.lse_out[static_cast<int64_t>(q0 + i) * a.hq + h] =
            l == 0.f ? -INFINITY : (mr + tc::log2_fast(l)) * kLn2;
    } else if (ok && real) {                             // (a tile none of whose rows sees a key)
      const int64_t at = static_cast<int64_t>(q0 + i) * a.hq + h;
      for (int c = 0; c < kNope / 8; ++c)
        reinterpret_cast<uint4*>(a.out + at * kNope)[c] = make_uint4(0, 0, 0, 0);
      if (a.lse_out != nullptr) a.lse_out[at] = -INFINITY;
    }
    if (!ok && lane == 0) raise_flag(a.flag, PKV_FLAG_TIMEOUT);
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMmaWarp) tc::tmem_free(tbase, kTmemCols);
}

cudaError_t launch_expanded(const ExpandedArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& rmap, const CUtensorMap& vmap, int num_sms,
                            cudaStream_t stream) {
  static DeviceSet done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!done.has(dev)) {
    e = cudaFuncSetAttribute(expanded_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(expanded_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    done.add(dev);
  }
  // (requests of 1 .. max_query_len tokens, num_tokens together)
  auto blocks = [&](int rows) {
    const int64_t requests = std::min<int64_t>(a.num_seqs, a.num_tokens);
    return std::min(requests * ((a.max_query_len - 1) / rows + 1),
                    (a.num_tokens + requests * (rows - 1)) / rows) * a.hq;
  };
  // One tile a block and its keys shared out, where two tiles a block would leave SMs idle,
  // or where no request has rows for a second one.  256 new tokens on 2048 keys, 16 heads (0.21
  // blocks of two tiles an SM): 22.0 us against 35.4; 2048 tokens, 16 heads (0.95): 30.1 against
  // 37.4; 1024 tokens, 32 heads (1.05): 23.2 against 23.1; 2048 tokens, 32 heads (1.89): 58.1
  // against 45.9, since keys are loaded twice as often; 128 tokens on 8192 keys, 128 heads:
  // 90.5 against 111.
  const bool halves = a.max_query_len <= kRows || blocks(2 * kRows) <= kFewUnits * num_sms;
  const int64_t grid = blocks(halves ? kRows : 2 * kRows);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return halves ? cudaLaunchKernelEx(&cfg, expanded_kernel<true>, qmap, kmap, rmap, vmap, a)
                : cudaLaunchKernelEx(&cfg, expanded_kernel<false>, qmap, kmap, rmap, vmap, a);
}

}  // namespace pkv
