// Attention over a 4-bit E2M1 cache: decode rows, and long requests in 16-row
// tiles where the tensor-core prefill does not apply.
//
// "Inside the engine: kernels, CUDA graphs and the life of a request":
// "Never materialise the TxT matrix" (online softmax), "Prefill has a full
// grid; decode at batch 1 has almost none" (split-KV partials, merged by the
// combine kernel) and "Attention over a block table, not a contiguous tensor".
//
// Mathematics.  With k = t_k s_k c_k and v = t_v s_v c_v (t a tensor's scale, s a
// block's E4M3 scale, c an E2M1 code), the products s c are f16 values, so both
// contractions run on mma.sync m16n8k16 with f16 operands over exactly what the
// cache holds; t_k joins the score scale and t_v the final 1 / l.  q rows enter
// as f16 scaled by a power of two per row (the row's largest magnitude in
// [2^14, 2^15); exact for every element within 2^31 of it).  p = 2^(x - m) is
// rounded to f16 for P V: the output divides by the sum of the rounded p (taken
// by one more MMA against ones), so it is an exact weighted average of V rows;
// the log-sum-exp uses the fp32 sum of p.
//
// Layout.  One CTA = (split, KV head, tile of 8 or 16 rows of one request); a
// row is (new token, query head of the group).  Both contractions are taken
// transposed (S^T = K Q^T, O^T = V^T P^T), so keys and output dims fill the MMA's
// 16 rows and the tile's rows its 8 columns.  Every warp streams its own pairs
// of 16-token blocks (32 keys) through its own ring of three cp.async stages: no
// barrier between warps until the merge.  A step computes the next pair's scores
// beside this pair's P V.
//   K: lane (g, q) holds key rows kappa(g) and kappa(g) + 8, and of each the
//   D / 4 consecutive elements at q D / 4: one 16-byte load of codes whose
//   bytes are MMA operand pairs in order, and its own two block scales.
//   V: lane (g, q) holds the D / 8 elements at g D / 8 (one block scale) of keys
//   q, (q ^ 1) + 4 and the same + 8, nibbles interleaved so a byte is the two
//   keys of an operand pair.
//   kappa(2 q) = q, kappa(2 q + 1) = (q ^ 1) + 4 makes the transposed score
//   fragment (movmatrix) the P^T operand of those V keys, keeps K's row loads
//   free of bank conflicts (D 128), and V's at two ways.
//
// What bounds it.  Bytes per (key, KV head): 2 x 9 D / 16.  Two contexts of 128K
// keys (302 MB, 32 / 8 heads of 128) take 58.4 us, 5.2 TB/s with the combine, 76% of
// the measured copy rate; the same loads without arithmetic 55 us.  64 requests
// of 512 to 4096 keys (169 MB) take 41.7 us, 42.5 with their new rows written in
// the same launch; their loads alone 32.  512 CTAs of unequal length share 304
// slots: a second wave begins with its table and first loads again, and by itself
// the launch leaves the SMs idle for a quarter of its time; while they run, 50% of the
// issue slots and 43% of the ALU pipe are taken (267 instructions a block and KV head:
// 64 code conversions, 64 scale products, 17 MMAs).  One request of 8192 keys takes
// 8.9 us: latency (metadata, table, first loads, 2 pairs a warp, merge, combine).
#include <cmath>

#include "device_set.h"
#include "e2m1.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B: 16x16 f16 A (rows g, g + 8; k 2q, 2q + 1 and + 8), 16x8 f16 B (column
// g), fp32 D (rows g: d0, d1; g + 8: d2, d3; columns 2q, 2q + 1)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 bytes to shared memory
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint8_t* p) {
  if constexpr (WORDS == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// p = 2^(x - ref) is kept below 2^(kSlack + kLift): the reference of a row moves
// only when a score passes it by more than kSlack + kLift, and it is set
// kLift below the row's maximum, so a row's largest p is at least 2^kLift and
// f16's subnormals (below 2^-14) start 2^21 under it.  A row without a score
// yet refers to the least float: its masked p are 0, and any finite score moves it.
constexpr float kSlack = 7.f, kLift = 7.f;
constexpr float kNoRef = -3.402823466e38f;

template <int D, int NT, int W>
struct Cfg {
  using P = E2m1Page<D>;
  static constexpr int kWarps = W;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = 8 * NT;
  using Stage = E2m1Stage<D>;
  static constexpr int kPair = Stage::kPair;
  static constexpr int kPairKeys = kPair * kBlock;
  static constexpr int kStageBytes = Stage::kBytes;
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMerge = kWarps * kRows * (D + 3) * 4;
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static constexpr int kCtas = W <= 6 ? 2 : 1;           // per SM
};

// What a CTA does for its request: the row tile's keys, and the blocks of its split.
struct TileRange {
  static constexpr int kRun = 0, kNothing = 1, kBad = 2;
  int state, splits;
  KeyRange keys;
};
__device__ __forceinline__ TileRange tile_range(const AttnArgs& a, int q0, int q1, int L, int split,
                                                int rho0, int rows_per_tile) {
  TileRange t = {TileRange::kNothing, 1, {0, 0, 0, 0}};
  const int n = q1 - q0;
  if (n == 0) return t;
  if (n < 0 || q0 < 0 || q1 > a.num_tokens || n > L || n > a.max_query_len ||
      L > static_cast<int64_t>(a.max_blocks_per_seq) * kBlock) {
    t.state = TileRange::kBad;
    return t;
  }
  const bool decode_class = n <= kDecodeMaxQ;
  if (!decode_class && (!a.long_rows || split > 0)) return t;   // (long requests are not split)
  const int rows_total = a.group * n;
  if (rho0 >= rows_total) return t;
  const int i_first = rho0 / a.group;
  const int i_last = (min(rho0 + rows_per_tile, rows_total) - 1) / a.group;
  t.state = TileRange::kRun;
  t.splits = decode_class ? a.num_splits : 1;
  t.keys = key_range(L, n, a.causal, a.window, i_first, i_last, t.splits, split);
  return t;
}

}  // namespace

template <int D, int NT, int W>
__global__ void __launch_bounds__(Cfg<D, NT, W>::kThreads, (Cfg<D, NT, W>::kCtas))
    decode_e2m1_kernel(const AttnArgs a) {
  using C = Cfg<D, NT, W>;
  using P = E2m1Page<D>;
  using Stage = E2m1Stage<D>;
  constexpr int kKWords = D / 32;                        // code words of a lane's K row part
  constexpr int kVWords = D / 64;                        // code words of a lane's V row part
  constexpr int kMT = D / 16;                            // 16-dim tiles of O^T, MMAs of a key block
  constexpr int R = C::kRows;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g8 = lane >> 2, t4 = lane & 3;

  const int kvh = static_cast<int>(blockIdx.x) % a.hkv;
  const int split = static_cast<int>(blockIdx.x) / a.hkv;
  const int rho0 = blockIdx.y * R;
  int r = blockIdx.z, q0, q1, L;
  // released only after the wait: a prefill behind this grid may count on
  // every input being complete
  pdl_wait_primary();
  pdl_launch_dependents();

  if (a.lpt) {
    r = request_by_length_rank(a, r, false, q0, q1, L);  // longest first
  } else {
    q0 = __ldg(a.qsl + r);
    q1 = __ldg(a.qsl + r + 1);
    L = __ldg(a.seq_lens + r);
  }
  const TileRange range = tile_range(a, q0, q1, L, split, rho0, R);
  if (range.state != TileRange::kRun) {
    if (range.state == TileRange::kBad && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
      raise_flag(a.flag, PKV_FLAG_BAD_LENGTHS);
    return;
  }
  const int group = a.group, n = q1 - q0;
  const int rows_total = group * n;
  const int nrows = min(R, rows_total - rho0);
  const int i_first = rho0 / group, i_last = (rho0 + nrows - 1) / group;
  const int splits = range.splits;
  const int kv_hi = range.keys.kv_hi, kv_lo = range.keys.kv_lo;
  const int b_end = range.keys.b_end;
  // keys every row of the tile sees: [in_lo, in_hi)
  const int in_hi = min(a.causal ? L - n + i_first + 1 : L, b_end * kBlock);
  const int in_lo = a.window > 0 ? max(0, L - n + i_last - a.window + 1) : 0;
  const int cap = min(kv_hi, b_end * kBlock);            // keys the split may see

  // ---- the warp's ring: pair u = warp + k * kWarps, k = 0, 1, ... ----
  uint8_t* const ring = smem + warp * (C::kStages * C::kStageBytes);
  uint8_t* const ring_end = ring + C::kStages * C::kStageBytes;
  const int32_t* table = a.block_table + static_cast<int64_t>(r) * a.max_blocks_per_seq;
  const int npw = warp_pairs(range.keys, warp, C::kWarps);
  const uint32_t page_stride = static_cast<uint32_t>(a.hkv) * P::kBytes;
  const uint8_t* kbase = static_cast<const uint8_t*>(a.k_cache) + kvh * P::kBytes;
  const uint8_t* vbase = static_cast<const uint8_t*>(a.v_cache) + kvh * P::kBytes;
  // this lane's chunk of the scale areas
  const bool has_scales = lane < Stage::kScaleLanes;
  const uint8_t* sbase =
      (Stage::scale_page(lane) < C::kPair ? kbase : vbase) + Stage::scale_source(lane);
  kbase += Stage::code_chunk(lane, 0);
  vbase += Stage::code_chunk(lane, 0);
  // table entries of 16 consecutive pairs of the warp, two a lane pair; 0 (a
  // page that exists) stands for a block past the run, whose keys are masked,
  // and for an entry outside the cache, whose rows are unspecified
  auto load_ids = [&](int k0) -> uint32_t {
    const int k = k0 + (lane >> 1);
    const int blk = pair_block(range.keys, warp, C::kWarps, k) + (lane & 1);
    if (k >= npw || blk >= b_end) return 0;
    const int32_t id = __ldg(table + blk);
    if (id < 0 || id >= a.num_blocks) {
      raise_flag(a.flag, PKV_FLAG_BAD_BLOCK);
      return 0;
    }
    return static_cast<uint32_t>(id);
  };
  // Fused write (decode steps): the CTA stores its KV head's rows of the new
  // tokens among the keys it reads, a scale block (of K or of V) a thread: loaded
  // here, stored once the pairs that hold no new token are on their way.  The
  // other pairs are loaded after that; a second row tile of a request stores the
  // same bytes.
  constexpr int kNewUnits = 2 * P::kRowScales;           // scale blocks of a token's K and V row
  static_assert(kDecodeMaxQ * kNewUnits <= C::kThreads, "a thread per scale block");
  const int new_lo = new_keys_lo(L, n, range.keys);
  const int new_hi = a.fuse_write ? new_keys_hi(range.keys) : 0;
  const bool stores = static_cast<int>(threadIdx.x) < (new_hi - new_lo) * kNewUnits;
  const int new_b = threadIdx.x % P::kRowScales;
  const bool new_v = (threadIdx.x / P::kRowScales) & 1;
  int64_t slot = -1;
  Raw16<__nv_bfloat16> raw;
  if (stores) {
    const int64_t t = q0 + new_lo - (L - n) + threadIdx.x / kNewUnits;
    slot = __ldg(a.slots + t);
    raw.load(static_cast<const __nv_bfloat16*>(new_v ? a.v_new : a.k_new) +
             (t * a.hkv + kvh) * D + new_b * kQuant);
  }
  uint32_t ids = load_ids(0);
  uint8_t* put = ring;                                   // the stage that is filled next
  auto issue = [&](int k) {
    if (k < npw) {
      if ((k & 15) == 0 && k > 0) ids = load_ids(k);
      const uint32_t to = smem_u32(put) + Stage::code_chunk(lane, 0);
#pragma unroll
      for (int j = 0; j < C::kPair; ++j) {
        const uint64_t off = static_cast<uint64_t>(__shfl_sync(0xffffffffu, ids, 2 * (k & 15) + j)) *
                             page_stride;
#pragma unroll
        for (int c = 0; c < Stage::kCodeChunks; ++c) {
          cp_async16(to + Stage::codes(0, j) + c * 512, kbase + off + c * 512);
          cp_async16(to + Stage::codes(1, j) + c * 512, vbase + off + c * 512);
        }
      }
      const uint32_t id = __shfl_sync(0xffffffffu, ids, 2 * (k & 15) + (Stage::scale_page(lane) & 1));
      if (has_scales)
        cp_async16(smem_u32(put) + Stage::scale_dest(lane), sbase + static_cast<uint64_t>(id) * page_stride);
      put += C::kStageBytes;
      if (put == ring_end) put = ring;
    }
    cp_async_commit();
  };
  const int early =                                      // the warp's first pair that has to wait
      new_lo < new_hi ? waiting_pair(range.keys, new_lo, warp, C::kWarps) : npw;
#pragma unroll
  for (int k = 0; k < C::kStages - 1; ++k)
    if (k < early) issue(k);
  if (new_lo < new_hi) {
    if (slot >= a.num_blocks * kBlock) {                 // outside the cache: skip, report
      raise_flag(a.flag, PKV_FLAG_BAD_SLOT);
    } else if (slot >= 0) {                              // (negative: padding)
      uint2 codes;
      uint32_t scale;
      const float t = new_v ? a.wv_scale : a.wk_scale;
      quantise16(raw, {t, __fdiv_rn(1.f, t)}, codes, scale);
      const int row = static_cast<int>(slot % kBlock);
      uint8_t* page = static_cast<uint8_t*>(const_cast<void*>(new_v ? a.v_cache : a.k_cache)) +
                      ((slot / kBlock) * a.hkv + kvh) * P::kBytes;
      *reinterpret_cast<uint2*>(page + row * P::kRowCodes + new_b * (kQuant / 2)) = codes;
      page[P::kCodes + row * P::kRowScales + new_b] = static_cast<uint8_t>(scale);
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < C::kStages - 1; ++k)
    if (k >= early) issue(k);

  // ---- this lane's q rows as f16 fragments, and its score columns' scales ----
  uint32_t qf[NT][kMT][2];
  float sc[NT][2];
  int lim[NT][2], low[NT][2];                            // visible keys of columns 2 t4, + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int rr = rho0 + 8 * nt + g8;
    uint32_t w[kMT * 2];
#pragma unroll
    for (int c = 0; c < kMT * 2; ++c) w[c] = 0;
    if (rr < rows_total) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(a.q) +
          (static_cast<int64_t>(q0 + rr / group) * a.hq + kvh * group + rr % group) * D +
          t4 * (D / 4));
#pragma unroll
      for (int c = 0; c < kMT / 2; ++c) {
        const uint4 v = __ldg(src + c);
        w[4 * c] = v.x;
        w[4 * c + 1] = v.y;
        w[4 * c + 2] = v.z;
        w[4 * c + 3] = v.w;
      }
    }
    uint32_t mx = 0;
#pragma unroll
    for (int c = 0; c < kMT * 2; ++c) mx = __vmaxu2(mx, w[c] & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const uint32_t m16 = max(mx & 0xFFFFu, mx >> 16);
    // largest |q| in [2^E, 2^(E+1)): e = E - 14 (clamped so 2^-e and 2^e are
    // normal floats; a zero row takes the lower bound)
    const int e = min(max(static_cast<int>(m16 >> 7) - 127 - 14, -100), 113);
    const float down =
        a.scale_log2 < 0.f ? -__int_as_float((127 - e) << 23) : __int_as_float((127 - e) << 23);
#pragma unroll
    for (int c = 0; c < kMT * 2; ++c)
      qf[nt][c >> 1][c & 1] = pack_f16x2(bf16_lo(w[c]) * down, bf16_hi(w[c]) * down);
    // (a positive score scale: its sign goes to q; at least the least normal
    // float, so that a masked -inf stays one)
    const float row_sc = fmaxf(fabsf(a.scale_log2) * __int_as_float((127 + e) << 23), 1.17549435e-38f);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      sc[nt][c] = __shfl_sync(0xffffffffu, row_sc, (2 * t4 + c) * 4);
      const int i = min(rho0 + 8 * nt + 2 * t4 + c, rows_total - 1) / group;
      lim[nt][c] = min(a.causal ? L - n + i + 1 : L, cap);
      low[nt][c] = a.window > 0 ? L - n + i - a.window + 1 : 0;
    }
  }

  const int ka = score_key(lane);                        // kappa(g8); the lane's other key + 8
  float oacc[NT][kMT][4];
  float ref[NT][2], l[NT][2], lr[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) oacc[nt][i][c] = 0.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ref[nt][c] = kNoRef;
      l[nt][c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) lr[nt][c] = 0.f;
  }

  // S^T (unscaled) of the pair in a stage
  float s[C::kPair][NT][4];
  auto scores = [&](const uint8_t* st, float (&x)[C::kPair][NT][4]) {
#pragma unroll
    for (int j = 0; j < C::kPair; ++j) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[j][nt][c] = 0.f;
      uint32_t wa[kKWords], wb[kKWords], sa[2], sb[2];
      const uint8_t* row = st + Stage::codes(0, j) + k_codes_at<D>(lane);
      load_words<kKWords>(wa, row);
      load_words<kKWords>(wb, row + 8 * P::kRowCodes);
      const uint8_t* srow = st + Stage::scales(0, j) + k_scales_at<D>(lane);
      if constexpr (D == 128) {
        const uint32_t ha = scales2_to_f16x2(*reinterpret_cast<const uint16_t*>(srow));
        const uint32_t hb =
            scales2_to_f16x2(*reinterpret_cast<const uint16_t*>(srow + 8 * P::kRowScales));
        sa[0] = byte_perm(ha, ha, 0x1010);
        sa[1] = byte_perm(ha, ha, 0x3232);
        sb[0] = byte_perm(hb, hb, 0x1010);
        sb[1] = byte_perm(hb, hb, 0x3232);
      } else {
        sa[0] = sa[1] = scales2_to_f16x2(srow[0] * 0x0101u);
        sb[0] = sb[1] = scales2_to_f16x2(srow[8 * P::kRowScales] * 0x0101u);
      }
#pragma unroll
      for (int w = 0; w < kKWords; ++w) {
        uint32_t ra[4], rb[4];
        e2m1x8_to_f16x2x4(wa[w], ra);
        e2m1x8_to_f16x2x4(wb[w], rb);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ra[c] = mul_f16x2(ra[c], sa[w >> 1]);
          rb[c] = mul_f16x2(rb[c], sb[w >> 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(x[j][nt], ra[0], rb[0], ra[1], rb[1], qf[nt][2 * w][0], qf[nt][2 * w][1]);
          mma_f16(x[j][nt], ra[2], rb[2], ra[3], rb[3], qf[nt][2 * w + 1][0],
                  qf[nt][2 * w + 1][1]);
        }
      }
    }
  };

  // Step k takes the scores of pair k, then its P V beside the scores of pair
  // k + 1: one run of independent work between two branches.
  const uint8_t* st = ring;                              // the stage of pair k
  if (npw > 0) {
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    scores(st, s);
  }
  for (int k = 0; k < npw; ++k) {
    issue(k + C::kStages - 1);                           // (into the stage that step k - 1 left)
    const int key0 = pair_block(range.keys, warp, C::kWarps, k) * kBlock;
    const bool edge = key0 + C::kPairKeys > in_hi || key0 < in_lo;
    // this lane's V scales: block g8 D / 128 of its four keys of both blocks
    uint32_t cs[C::kPair][4];
#pragma unroll
    for (int j = 0; j < C::kPair; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        cs[j][c] = st[Stage::scales(1, j) + v_scales_at<D>(lane, c)];
    if (edge) {
      // p is 0 outside a row's keys, and so must p v be whatever a hidden slot
      // holds: a scale outside the tile's keys, or a NaN one that some row of
      // the tile may not see, counts as 0 (a 0 code times any finite scale)
      bool bad = false;
#pragma unroll
      for (int j = 0; j < C::kPair; ++j) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = key0 + j * kBlock + ka + (c >> 1) * 8;
            if (key >= lim[nt][c & 1] || key < low[nt][c & 1]) s[j][nt][c] = -INFINITY;
          }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = key0 + j * kBlock + value_key(lane, c);
          const bool nan = (cs[j][c] & 0x7F) == 0x7F;
          const bool in = key < cap && key >= kv_lo;
          bad = bad || (nan && in);
          if (nan || !in) cs[j][c] = 0;
          if (nan && in) cs[j][c] = 0x100;               // remembered below
        }
      }
      if (__any_sync(0xffffffffu, bad)) {
        // rows that do see such a key take the NaN in its block's dims
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int jc = 0; jc < 4 * C::kPair; ++jc) {
            const int j = jc / 4, c = jc % 4;
            const uint32_t v = __shfl_sync(0xffffffffu, cs[j][c], g8 * 4 + q);
            const int key = key0 + j * kBlock + value_key(q, c);
            if (v == 0x100) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (key < lim[nt][e] && key >= low[nt][e]) {
#pragma unroll
                    for (int i = 0; i < kMT; ++i)
                      oacc[nt][i][e] = oacc[nt][i][e + 2] = __int_as_float(0x7FC00000);
                  }
            }
          }
#pragma unroll
        for (int jc = 0; jc < 4 * C::kPair; ++jc) cs[jc / 4][jc % 4] &= 0xFF;
      }
    }
    uint32_t vs[C::kPair][2];
#pragma unroll
    for (int j = 0; j < C::kPair; ++j) {
      vs[j][0] = scales2_to_f16x2(cs[j][0] | (cs[j][1] << 8));
      vs[j][1] = scales2_to_f16x2(cs[j][2] | (cs[j][3] << 8));
    }
    // move a row's reference when a score passes it by kSlack + kLift
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx[2];
      bool up = false;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
        mx[c] *= sc[nt][c];
        up = up || mx[c] > ref[nt][c] + (kSlack + kLift);
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
            mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], o));
          if (mx[c] > ref[nt][c] + (kSlack + kLift)) {
            const float to = mx[c] - kLift;
            const float f = ex2(ref[nt][c] - to);        // (0 from kNoRef)
            ref[nt][c] = to;
            l[nt][c] *= f;
            lr[nt][c] *= f;
            lr[nt][c + 2] *= f;
#pragma unroll
            for (int i = 0; i < kMT; ++i) {
              oacc[nt][i][c] *= f;
              oacc[nt][i][c + 2] *= f;
            }
          }
        }
      }
    }
    // every lane's part of pair k + 1 has landed
    cp_async_wait<C::kStages - 2>();
    __syncwarp();
    // p, its sums, and P^T operands
    uint32_t pf[C::kPair][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < C::kPair; ++j) {
        float p[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          p[c] = ex2(fmaf(s[j][nt][c], sc[nt][c & 1], -ref[nt][c & 1]));
          l[nt][c & 1] += p[c];
        }
        pf[j][nt][0] = movmatrix_t(pack_f16x2(p[0], p[1]));
        pf[j][nt][1] = movmatrix_t(pack_f16x2(p[2], p[3]));
        // the sums of the rounded p: against a V of ones
        mma_f16(lr[nt], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pf[j][nt][0],
                pf[j][nt][1]);
      }
    }
    // (the scores of pair k + 1; past the warp's last pair, of an old stage)
    const uint8_t* next = st + C::kStageBytes == ring_end ? ring : st + C::kStageBytes;
    scores(next, s);
    // O^T += V^T P^T
#pragma unroll
    for (int j = 0; j < C::kPair; ++j) {
      const uint8_t* vrow = st + Stage::codes(1, j);
      uint32_t vw[4][kVWords];
#pragma unroll
      for (int c = 0; c < 4; ++c) load_words<kVWords>(vw[c], vrow + v_codes_at<D>(lane, c));
      const uint32_t s01 = vs[j][0], s23 = vs[j][1];
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        // byte i of e: element 2 i of both keys of a pair; of o: element 2 i + 1
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        uint32_t e01[4], o01[4], e23[4], o23[4];
        e2m1x8_to_f16x2x4((vw[0][w] & kLow) | ((vw[1][w] << 4) & ~kLow), e01);
        e2m1x8_to_f16x2x4(((vw[0][w] >> 4) & kLow) | (vw[1][w] & ~kLow), o01);
        e2m1x8_to_f16x2x4((vw[2][w] & kLow) | ((vw[3][w] << 4) & ~kLow), e23);
        e2m1x8_to_f16x2x4(((vw[2][w] >> 4) & kLow) | (vw[3][w] & ~kLow), o23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = mul_f16x2(e01[i], s01), a1 = mul_f16x2(o01[i], s01);
          const uint32_t a2 = mul_f16x2(e23[i], s23), a3 = mul_f16x2(o23[i], s23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(oacc[nt][4 * w + i], a0, a1, a2, a3, pf[j][nt][0], pf[j][nt][1]);
        }
      }
    }
    st = next;
    __syncwarp();                                        // the stage is read; step k + 1 refills it
  }
  cp_async_wait<0>();
  __syncthreads();                                       // every ring is idle: reuse for the merge

  // ---- merge of the warps' (ref, l, acc) ----
  float* mw = reinterpret_cast<float*>(smem);            // [warp][row]
  float* lw = mw + C::kWarps * R;
  float* lrw = lw + C::kWarps * R;
  float* aw = lrw + C::kWarps * R;                       // [warp][row][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float lt = l[nt][c];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
      const int rho = 8 * nt + 2 * t4 + c;
      if (g8 == 0) {
        mw[warp * R + rho] = ref[nt][c];
        lw[warp * R + rho] = lt;
        lrw[warp * R + rho] = lr[nt][c];
      }
      // 16-byte chunks of the row, permuted so that the 8 lanes of a store phase
      // (two g8, four rows) hit distinct banks
      if (rho < nrows) {
        float4* row = reinterpret_cast<float4*>(aw + (warp * R + rho) * D);
#pragma unroll
        for (int i = 0; i < kMT; i += 2)
          row[merge_chunk<D>(rho, g8 * (D / 32) + i / 2)] =
              make_float4(oacc[nt][i][c], oacc[nt][i][c + 2], oacc[nt][i + 1][c],
                          oacc[nt][i + 1][c + 2]);
      }
    }
  __syncthreads();
  constexpr int kDPL = D / 32;
  for (int rho = warp; rho < nrows; rho += C::kWarps) {
    float M = kNoRef;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) M = fmaxf(M, mw[w * R + rho]);
    float o[kDPL];
#pragma unroll
    for (int e = 0; e < kDPL; ++e) o[e] = 0.f;
    float lsum = 0.f, lnorm = 0.f;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      const float f = ex2(mw[w * R + rho] - M);
      lsum = fmaf(f, lw[w * R + rho], lsum);
      lnorm = fmaf(f, lrw[w * R + rho], lnorm);
      const int chunk = merge_chunk<D>(rho, lane * kDPL / 4);
      const float* src = aw + (w * R + rho) * D + chunk * 4 + lane * kDPL % 4;
#pragma unroll
      for (int e = 0; e < kDPL; ++e) o[e] = fmaf(f, src[e], o[e]);
    }
    // (a NaN sum stays a NaN: only a row without a key takes 0)
    const float inv = lnorm == 0.f ? 0.f : a.v_scale / lnorm;
    const float lse2 = lsum == 0.f ? -INFINITY : M + lg2(lsum);
    const int rr = rho0 + rho, i = rr / group, h = kvh * group + rr % group;
    if (splits > 1) {
      const int64_t w =
          ((static_cast<int64_t>(split) * a.num_seqs + r) * kDecodeMaxQ + i) * a.hq + h;
      float* dst = a.ws_o + w * D + lane * kDPL;
      if constexpr (kDPL == 4)
        *reinterpret_cast<float4*>(dst) =
            make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
      else
        *reinterpret_cast<float2*>(dst) = make_float2(o[0] * inv, o[1] * inv);
      if (lane == 0) a.ws_lse[w] = lse2;
    } else {
      const int64_t t = q0 + i;
      __nv_bfloat16* dst =
          static_cast<__nv_bfloat16*>(a.out) + (t * a.hq + h) * D + lane * kDPL;
      if constexpr (kDPL == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
      if (a.lse_out != nullptr && lane == 0) a.lse_out[t * a.hq + h] = lse2 * kLn2;
    }
  }
}

template <int D, int NT, int W>
static cudaError_t launch_t(const AttnArgs& a, int row_tiles, cudaStream_t stream) {
  using C = Cfg<D, NT, W>;
  static DeviceSet done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!done.has(dev)) {
    e = cudaFuncSetAttribute(decode_e2m1_kernel<D, NT, W>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decode_e2m1_kernel<D, NT, W>,
                               cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    done.add(dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.hkv * a.num_splits),
                     static_cast<unsigned>(row_tiles), static_cast<unsigned>(a.num_seqs));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_e2m1_kernel<D, NT, W>, a);
}

// Rows per tile.  8 where that holds a request's rows; else 16, whose tiles read
// the cached rows once for all of them, unless the batch (seq_heads requests x KV
// heads, of nblk blocks) is too small for its 16-row tiles to fill the SMs at 32
// blocks a CTA: then 8-row tiles share out the latency.  Measured, us, 16 / 8
// rows: 16 requests of 3 tokens, 16 query heads to one KV head, 1027 keys 13.0 /
// 10.3; one request of 8192 keys, so headed, 9.2 / 7.5; 16 requests of 4 tokens,
// 32 / 8 heads, 2048 keys 19.7 / 21.5; 64 requests, 32 / 2 heads, 4096 keys 30.9 /
// 35.7.  Beside requests that the prefill kernel takes (max_query_len above the
// decode bound, no long_rows), the decode rows are taken to be single tokens, as
// such batches have them.
int decode_e2m1_rows_per_tile(int group, int max_query_len, bool long_rows, int64_t seq_heads,
                              int64_t nblk, int num_sms) {
  const int64_t q = long_rows                     ? max_query_len
                    : max_query_len > kDecodeMaxQ ? 1
                                                  : max_query_len;
  const int64_t rows = group * (q < 1 ? 1 : q);
  if (rows <= 8) return 8;
  if (long_rows) return 16;
  const int64_t ctas = seq_heads * ((rows + 15) / 16) * (nblk < 32 ? 1 : nblk / 32);
  return ctas <= num_sms ? 8 : 16;
}

// Warps per CTA: 8-row tiles run two CTAs of 6 on an SM, or one of 8 where the
// grid does not give every SM a second one; 16-row tiles (up to 232 registers a
// thread) one of 8.  A warp alone takes about 2000 cycles a pair of blocks, so
// what a lone CTA's warps share out counts, against the merge of more warps: one
// request over 8 KV heads takes, with 6 / 8 / 12 warps, 6.3 / 6.2 / 6.7 us for 512
// keys (1 split), 7.9 / 7.5 / 7.8 for 4096 (16) and 19.8 / 15.9 / 16.6 for 32768
// (19).  12 warps in two CTAs an SM are as fast as 16 (the long cases are bound
// by HBM), and three CTAs of 4 slower.
constexpr int kWarps8 = 6, kWarps8Lone = 8, kWarps16 = 8;

// Resident CTAs per SM for that tile height.
int decode_e2m1_ctas_per_sm(int rows_per_tile) {
  return rows_per_tile == 8 ? Cfg<128, 1, kWarps8>::kCtas : Cfg<128, 2, kWarps16>::kCtas;
}

template <int D>
static cudaError_t launch_d(const AttnArgs& a, int rows_per_tile, int row_tiles, int num_sms,
                            cudaStream_t stream) {
  if (rows_per_tile != 8) return launch_t<D, 2, kWarps16>(a, row_tiles, stream);
  const int64_t ctas = static_cast<int64_t>(a.hkv) * a.num_splits * row_tiles * a.num_seqs;
  return ctas <= num_sms ? launch_t<D, 1, kWarps8Lone>(a, row_tiles, stream)
                         : launch_t<D, 1, kWarps8>(a, row_tiles, stream);
}

cudaError_t launch_decode_e2m1(const AttnArgs& a, int head_dim, int num_sms,
                               cudaStream_t stream) {
  const int span = a.window > 0 && a.window < a.max_seq_len - kDecodeMaxQ
                       ? a.window + kDecodeMaxQ : a.max_seq_len;
  const int R = decode_e2m1_rows_per_tile(a.group, a.max_query_len, a.long_rows != 0,
                                          static_cast<int64_t>(a.num_seqs) * a.hkv,
                                          (static_cast<int64_t>(span) + kBlock - 1) / kBlock, num_sms);
  const int64_t q = a.long_rows || a.max_query_len < kDecodeMaxQ ? a.max_query_len : kDecodeMaxQ;
  const int64_t row_tiles = (a.group * q + R - 1) / R;
  if (row_tiles < 1 || row_tiles > 65535 || a.num_seqs > 65535)
    return cudaErrorInvalidConfiguration;
  const int tiles = static_cast<int>(row_tiles);
  return head_dim == 128 ? launch_d<128>(a, R, tiles, num_sms, stream)
                         : launch_d<64>(a, R, tiles, num_sms, stream);
}

}  // namespace pkv
