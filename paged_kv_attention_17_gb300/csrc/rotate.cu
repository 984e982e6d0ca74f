// Position rotation of a step's queries and keys, with the keys and values
// appended to their cache: the rotated form of the slot-mapped write, and the
// write of a latent cache.
//
// "Model execution", section "Flattening a step": positions name each new token's
// place in its request, slot_mapping the cache slot of its K and V.  The rotation
// turns pair i of a head's leading elements by t = position * inv_freq[i],
//   y_a = a cos t - b sin t,   y_b = a sin t + b cos t,
// (a, b) the elements i and i + rotary_dim / 2, or 2 i and 2 i + 1 (interleaved).
// With several axes (time, height, width) each pair goes by one axis's position.
//
// The angle.  t is needed modulo a turn only, and a far position times a
// frequency has no fp32 product exact enough (131071 rad: half an ulp is 0.004).
// So frequencies are taken as 64-bit fractions of a turn, whose product with an
// integer position wraps modulo 2^64, that is modulo whole turns, by itself: the
// fraction is off by 2^-53 of itself, the angle by |t| 2^-53 and the 2^-32 turns
// that its top word drops, then rounded once to fp32.
//
// Both rows of a pair, and a whole pair of 16-byte chunks, belong to one thread (a
// unit), so q may be turned in place.  A block takes a group of tokens at a time; their
// angles' sines and cosines are computed once a token, in shared memory, and serve every
// head.  A thread's units are the same in every group, so where they lie is worked out
// once; the next group's rows are on their way while this one's are turned.  HBM bounds
// it: bytes per token are the rows of q (read and written), k and v (read, and written in
// the cache's type).  8192 tokens of 32 and 8 heads of 128 in bf16, 201 MB, take 40 us (5.0
// TB/s; a plain copy of as many bytes takes 37), in fp32, 403 MB, 70 us (5.8 TB/s), 8192 latent
// rows with 32 heads' q, 86 MB, 24 us (a copy 20).  Into caches of codes the instructions weigh
// more than the bytes saved: E4M3, 185 MB, 47 us (3.9 TB/s; 1.4 times the instructions of bf16,
// issue slots 48% taken, loads one group ahead), E2M1, 177 MB, 49 us (3.6 TB/s; 1.7 times,
// 55%, the ALU pipe 53%, and a block that takes one group has nothing under way at its ends).
#include <algorithm>

#include "common.cuh"
#include "e2m1.cuh"
#include "rotate.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroup = 8;                     // tokens of a block
constexpr int kUnits = 3;                        // units of a thread, of a long batch

// inv_freq (radians a position) as a 64-bit fraction of a turn.  With f = m 2^e, m
// of 24 bits, and K = 2^66 / (2 pi) in 64 bits (53 of them exact), it is the low 64
// bits of m K 2^(e - 2).
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr double kInvTurn = 0.15915494309189535;               // 1 / (2 pi)
  constexpr uint64_t kK = static_cast<uint64_t>(kInvTurn * 4.0 * 18446744073709551616.0);
  const uint32_t bits = __float_as_uint(f);
  const int exp = static_cast<int>((bits >> 23) & 0xFF);
  const uint64_t m = exp == 0 ? (bits & 0x7FFFFFu) : ((bits & 0x7FFFFFu) | 0x800000u);
  const uint64_t lo = m * kK, hi = __umul64hi(m, kK);
  const int right = 152 - (exp == 0 ? 1 : exp);                  // places, of the 128 bits
  uint64_t v;
  if (right >= 64)
    v = right >= 128 ? 0 : hi >> (right - 64);
  else if (right > 0)
    v = (lo >> right) | (hi << (64 - right));
  else
    v = -right >= 64 ? 0 : lo << -right;
  return (bits >> 31) != 0 ? 0 - v : v;
}

// (cos, sin) of position * f, f a fraction of a turn
__device__ __forceinline__ float2 turn(int64_t position, uint64_t f) {
  const uint64_t phase = static_cast<uint64_t>(position) * f;
  const float half_turns = __int2float_rn(static_cast<int>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// The angles of a group lie in shared memory, pair after pair of a token; two pairs' room is
// left behind every eight, so that threads of neighbouring units read distinct banks.
__host__ __device__ constexpr int angle_at(int pair) { return pair + pair / 8 * 2; }
__host__ __device__ constexpr int angles_of(int rotary) { return (angle_at(rotary / 2 - 1) + 2) / 2 * 2; }
static_assert(angles_of(16) % 2 == 0 && angles_of(64) % 2 == 0 && angles_of(1024) % 2 == 0 &&
                  2 * angles_of(1024) * 8 <= 49152, "16-byte rows of angles, a token at least");

// One thread's angle of a group: token t, pair p of it, with the fraction of p worked out and
// the position loaded ahead.
struct Angle {
  int t, p;
  uint64_t fraction;
  const int64_t* position;
  int64_t next;
  __device__ __forceinline__ Angle(const RotateArgs& a, int i) {
    const int pairs = a.rotary / 2;
    t = i / pairs;
    p = i - t * pairs;
    int axis = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) axis += p >= a.section_end[k] ? 1 : 0;
    position = a.positions + axis * a.num_tokens + t;
    fraction = t < a.group ? turn_fraction(__ldg(a.inv_freq + p)) : 0;
  }
  __device__ __forceinline__ void fetch(const RotateArgs& a, int64_t t0) {
    if (t < a.group && t0 + t < a.num_tokens) next = __ldg(position + t0);
  }
  __device__ __forceinline__ void fill(const RotateArgs& a, int64_t t0, float2* angles) const {
    if (t < a.group && t0 + t < a.num_tokens)
      angles[t * angles_of(a.rotary) + angle_at(p)] = turn(next, fraction);
  }
};
// The angles of a group behind the first kThreads.
__device__ __forceinline__ void fill_rest(const RotateArgs& a, int64_t t0, float2* angles) {
  for (int i = threadIdx.x + kThreads; i < a.group * (a.rotary / 2); i += kThreads) {
    Angle x(a, i);
    x.fetch(a, t0);
    x.fill(a, t0, angles);
  }
}

template <typename S>
struct Chunk {                                   // 16 bytes of a row
  static constexpr int kN = 16 / static_cast<int>(sizeof(S));
  static __device__ __forceinline__ void widen(const uint4& w, float (&f)[kN]) {
    if constexpr (sizeof(S) == 4) {
      f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
      f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    } else {
      f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
      f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[kN]) {
    uint4 w;
    if constexpr (sizeof(S) == 4) {
      w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
    } else {
      __nv_bfloat162 p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w = *reinterpret_cast<const uint4*>(p);
    }
    return w;
  }
};

// A turned pair, c = (cos, sin); the roundings spelt out, so that every cache type
// holds codes of the same fp32 values.
__device__ __forceinline__ float turned_a(float a, float b, float2 c) {
  return fmaf(a, c.x, -__fmul_rn(b, c.y));
}
__device__ __forceinline__ float turned_b(float a, float b, float2 c) {
  return fmaf(a, c.y, __fmul_rn(b, c.x));
}

// Turn N pairs held in two runs of N elements: pairs (x[i], y[i]), or interleaved
// (elements 2 i and 2 i + 1 of x followed by y).  angles: of the token; `first`, a multiple
// of N, is the first pair.
template <int N>
__device__ __forceinline__ void turn_pairs(float (&x)[N], float (&y)[N], const float2* angles,
                                           int first, bool interleaved) {
  float2 c[N];
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float4 w = *reinterpret_cast<const float4*>(angles + angle_at(first + i));
    c[i] = make_float2(w.x, w.y);
    c[i + 1] = make_float2(w.z, w.w);
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 u = c[i], w = c[N / 2 + i];
      const float a = x[2 * i], b = x[2 * i + 1], e = y[2 * i], f = y[2 * i + 1];
      x[2 * i] = turned_a(a, b, u);
      x[2 * i + 1] = turned_b(a, b, u);
      y[2 * i] = turned_a(e, f, w);
      y[2 * i + 1] = turned_b(e, f, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float a = x[i], b = y[i];
      x[i] = turned_a(a, b, c[i]);
      y[i] = turned_b(a, b, c[i]);
    }
  }
}

// A unit of a head's row of `dim` elements, as two runs of N consecutive elements:
// turned units pair the runs u and u + rotary / 2 / N, or interleaved 2 u and 2 u + 1;
// the units behind them are plain runs 2 u and 2 u + 1.  (rotary is a multiple of 2 N.)
template <int N>
struct Unit {
  int first, second, pair;                       // elements; the first pair, -1: not turned
  __device__ __forceinline__ Unit(int u, int rotary, bool interleaved) {
    const int turned = rotary / (2 * N);
    const bool split = u < turned && !interleaved;
    first = split ? u * N : 2 * u * N;
    second = split ? (u + turned) * N : first + N;
    pair = u < turned ? u * N : -1;
  }
};

enum class Part { kQ, kK, kV };

// What one unit of a token's row stands for, and where.
struct Place {
  Part part;
  int head, unit;
};
__device__ __forceinline__ Place place_of(int u, int q_units, int k_units, int per_q, int per_k,
                                          int per_v) {
  Place p;
  p.part = u < q_units ? Part::kQ : (u < q_units + k_units ? Part::kK : Part::kV);
  u -= p.part == Part::kQ ? 0 : (p.part == Part::kK ? q_units : q_units + k_units);
  const int per = p.part == Part::kQ ? per_q : (p.part == Part::kK ? per_k : per_v);
  p.head = u / per;
  p.unit = u - p.head * per;
  return p;
}

// A token's slot, -1 where its rows are not stored.
__device__ __forceinline__ int64_t slot_of(const RotateArgs& a, int64_t t, bool tell) {
  const int64_t slot = __ldg(a.slots + t);
  if (slot < a.num_slots) return slot < 0 ? -1 : slot;
  if (tell) raise_flag(a.flag, PKV_FLAG_BAD_SLOT);
  return -1;
}

}  // namespace

// Caches of the rows' own type (E4M3 = false) or of 8-bit codes.  A group is a.group tokens;
// block (x, y) takes part y of the units of groups x, x + gridDim.x, ..., K a thread.
template <typename S, bool E4M3, int K>
__global__ void __launch_bounds__(kThreads, 2) rotate_write_kernel(const RotateArgs a) {
  constexpr int kN = Chunk<S>::kN;
  extern __shared__ __align__(16) float2 angles[];                     // two groups'
  pdl_launch_dependents();
  const int per = a.dim / (2 * kN), per_v = a.v_dim / (2 * kN);
  const int q_units = a.hq * per, k_units = a.hk * per, all = q_units + k_units + a.hv * per_v;
  const int64_t groups = (a.num_tokens + a.group - 1) / a.group;
  // this thread's units: the token of the group (-1: none), what, and where
  int token[K], pair[K], second[K];
  Part part[K];
  int64_t from[K], to[K];                                // q: q_out's element; else the slot's
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int i = (blockIdx.y * K + j) * kThreads + threadIdx.x;
    token[j] = i < a.group * all ? i / all : -1;
    const Place p = place_of(i % all, q_units, k_units, per, per, per_v);
    const Unit<kN> u(p.unit, p.part == Part::kV ? 0 : a.rotary, a.interleaved != 0);
    part[j] = p.part;
    pair[j] = u.pair;
    second[j] = u.second - u.first;
    const bool q = p.part == Part::kQ, v = p.part == Part::kV;
    from[j] = p.head * (q ? a.q_hs : v ? a.v_hs : a.k_hs) + u.first;
    to[j] = p.head * (q ? a.qo_hs : v ? static_cast<int64_t>(a.v_dim) : a.dim) + u.first;
  }
  auto load = [&](int64_t group, uint4 (&x)[K], uint4 (&y)[K]) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int64_t t = group * a.group + token[j];
      if (token[j] < 0 || t >= a.num_tokens) continue;
      const S* row = (part[j] == Part::kQ   ? static_cast<const S*>(a.q) + t * a.q_ts
                      : part[j] == Part::kK ? static_cast<const S*>(a.k) + t * a.k_ts
                                            : static_cast<const S*>(a.v) + t * a.v_ts) + from[j];
      x[j] = __ldcs(reinterpret_cast<const uint4*>(row));
      y[j] = __ldcs(reinterpret_cast<const uint4*>(row + second[j]));
    }
  };
  pdl_wait_primary();
  uint4 x[K], y[K];
  int64_t group = blockIdx.x;                            // (the grid has no more blocks)
  Angle angle(a, threadIdx.x);
  angle.fetch(a, group * a.group);
  load(group, x, y);
  float2* now = angles;
  float2* then = angles + a.group * angles_of(a.rotary);
  angle.fill(a, group * a.group, now);
  fill_rest(a, group * a.group, now);
  __syncthreads();
  while (true) {
    const int64_t next = group + gridDim.x;
    uint4 nx[K], ny[K];
    if (next < groups) {
      angle.fetch(a, next * a.group);
      load(next, nx, ny);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int64_t t = group * a.group + token[j];
      if (token[j] < 0 || t >= a.num_tokens) continue;
      const bool q = part[j] == Part::kQ, v = part[j] == Part::kV;
      float f[kN], g[kN];
      if (pair[j] >= 0 || (E4M3 && !q)) {
        Chunk<S>::widen(x[j], f);
        Chunk<S>::widen(y[j], g);
      }
      if (pair[j] >= 0) {
        turn_pairs<kN>(f, g, now + token[j] * angles_of(a.rotary), pair[j], a.interleaved != 0);
        if (!E4M3 || q) {
          x[j] = Chunk<S>::narrow(f);
          y[j] = Chunk<S>::narrow(g);
        }
      }
      if (q) {
        S* row = static_cast<S*>(a.q_out) + t * a.qo_ts + to[j];
        *reinterpret_cast<uint4*>(row) = x[j];
        *reinterpret_cast<uint4*>(row + second[j]) = y[j];
        continue;
      }
      const int64_t slot = slot_of(a, t, v && to[j] == 0);
      if (slot < 0) continue;
      const int64_t at = slot * (v ? a.vc_row : a.kc_row) + to[j];
      if constexpr (E4M3) {
        const float scale = v ? a.v_scale : a.k_scale;
        uint8_t* row = static_cast<uint8_t*>(v ? a.v_cache : a.k_cache) + at;
        uint32_t c[kN / 2], d[kN / 2];
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) {
          c[e] = float2_to_e4m3x2(__fdiv_rn(f[2 * e], scale), __fdiv_rn(f[2 * e + 1], scale));
          d[e] = float2_to_e4m3x2(__fdiv_rn(g[2 * e], scale), __fdiv_rn(g[2 * e + 1], scale));
        }
#pragma unroll
        for (int e = 0; e < kN / 4; ++e) {
          reinterpret_cast<uint32_t*>(row)[e] = c[2 * e] | (c[2 * e + 1] << 16);
          reinterpret_cast<uint32_t*>(row + second[j])[e] = d[2 * e] | (d[2 * e + 1] << 16);
        }
      } else {
        S* row = static_cast<S*>(v ? a.v_cache : a.k_cache) + at;
        *reinterpret_cast<uint4*>(row) = x[j];
        *reinterpret_cast<uint4*>(row + second[j]) = y[j];
      }
    }
    if (next >= groups) break;
    angle.fill(a, next * a.group, then);
    fill_rest(a, next * a.group, then);
    __syncthreads();                                     // (and this group's angles are read)
    float2* const swap = now;
    now = then;
    then = swap;
    group = next;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      x[j] = nx[j];
      y[j] = ny[j];
    }
  }
}

// 4-bit caches: a unit of k or v is two scale blocks of 16 elements (turned pairs are
// whole blocks apart), quantised from the turned fp32 values; q as above.
template <typename S>
__global__ void __launch_bounds__(kThreads, 2) rotate_write_e2m1_kernel(const RotateArgs a,
                                                                        const Divisor kd,
                                                                        const Divisor vd) {
  constexpr int kN = Chunk<S>::kN;
  extern __shared__ __align__(16) float2 angles[];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.group;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.group), a.num_tokens - t0));
  const int per = a.dim / (2 * kN), per_c = a.dim / (2 * kQuant);
  const int q_units = a.hq * per, k_units = a.hk * per_c, all = q_units + 2 * k_units;
  const int units = tokens * all;
  // (a unit's rows are loaded while the one before is turned and quantised)
  constexpr int kWords = static_cast<int>(sizeof(S));    // 16-byte words of 16 elements
  struct Ahead {
    int64_t t, slot;
    Place p;
    uint4 w[2 * kWords];
  };
  auto fetch = [&](int i, Ahead& n) {
    const int tt = i / all;
    n.t = t0 + tt;
    n.p = place_of(i - tt * all, q_units, k_units, per, per_c, per_c);
    if (n.p.part == Part::kQ) {
      const Unit<kN> u(n.p.unit, a.rotary, a.interleaved != 0);
      const S* row = static_cast<const S*>(a.q) + n.t * a.q_ts + n.p.head * a.q_hs;
      n.w[0] = __ldcs(reinterpret_cast<const uint4*>(row + u.first));
      n.w[1] = __ldcs(reinterpret_cast<const uint4*>(row + u.second));
      return;
    }
    const bool is_v = n.p.part == Part::kV;
    n.slot = __ldg(a.slots + n.t);
    const Unit<kQuant> u(n.p.unit, is_v ? 0 : a.rotary, a.interleaved != 0);
    const S* row = is_v ? static_cast<const S*>(a.v) + n.t * a.v_ts + n.p.head * a.v_hs
                        : static_cast<const S*>(a.k) + n.t * a.k_ts + n.p.head * a.k_hs;
#pragma unroll
    for (int e = 0; e < kWords; ++e) {
      n.w[e] = __ldcs(reinterpret_cast<const uint4*>(row + u.first) + e);
      n.w[kWords + e] = __ldcs(reinterpret_cast<const uint4*>(row + u.second) + e);
    }
  };
  const int step = kThreads * static_cast<int>(gridDim.y);
  int i = blockIdx.y * kThreads + threadIdx.x;
  Ahead ahead;
  if (i < units) fetch(i, ahead);
  Angle angle(a, threadIdx.x);
  angle.fetch(a, t0);
  angle.fill(a, t0, angles);
  fill_rest(a, t0, angles);
  __syncthreads();
  for (; i < units; i += step) {
    const Ahead now = ahead;
    if (i + step < units) fetch(i + step, ahead);
    const Place p = now.p;
    const float2* cs = angles + (now.t - t0) * angles_of(a.rotary);
    if (p.part == Part::kQ) {
      const Unit<kN> u(p.unit, a.rotary, a.interleaved != 0);
      S* to = static_cast<S*>(a.q_out) + now.t * a.qo_ts + p.head * a.qo_hs;
      uint4 x = now.w[0], y = now.w[1];
      if (u.pair >= 0) {
        float f[kN], g[kN];
        Chunk<S>::widen(x, f);
        Chunk<S>::widen(y, g);
        turn_pairs<kN>(f, g, cs, u.pair, a.interleaved != 0);
        x = Chunk<S>::narrow(f);
        y = Chunk<S>::narrow(g);
      }
      *reinterpret_cast<uint4*>(to + u.first) = x;
      *reinterpret_cast<uint4*>(to + u.second) = y;
      continue;
    }
    const bool is_v = p.part == Part::kV;
    const int64_t slot = now.slot;
    if (slot < 0) continue;
    if (slot >= a.num_slots) {
      if (is_v && p.head == 0 && p.unit == 0) raise_flag(a.flag, PKV_FLAG_BAD_SLOT);
      continue;
    }
    const Unit<kQuant> u(p.unit, is_v ? 0 : a.rotary, a.interleaved != 0);
    Raw16<S> r0, r1;
#pragma unroll
    for (int e = 0; e < kWords; ++e) {
      r0.w[e] = now.w[e];
      r1.w[e] = now.w[kWords + e];
    }
    uint8_t* page = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) +
                    ((slot / kBlock) * a.hk + p.head) * (9 * static_cast<int64_t>(a.dim));
    const int at = static_cast<int>(slot % kBlock);
    auto store = [&](int e, uint2 codes, uint32_t scale) {
      *reinterpret_cast<uint2*>(page + at * (a.dim / 2) + e / 2) = codes;
      page[8 * a.dim + at * (a.dim / kQuant) + e / kQuant] = static_cast<uint8_t>(scale);
    };
    uint2 codes;
    uint32_t scale;
    if (u.pair >= 0) {
      float f[kQuant], g[kQuant];
      r0.floats(f);
      r1.floats(g);
      turn_pairs<kQuant>(f, g, cs, u.pair, a.interleaved != 0);
      Raw16<float> w;
      auto pack = [&](const float (&v)[kQuant]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w.w[e] = make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                              __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
      };
      pack(f);
      quantise16(w, kd, codes, scale);
      store(u.first, codes, scale);
      pack(g);
      quantise16(w, kd, codes, scale);
      store(u.second, codes, scale);
    } else {
      quantise16(r0, is_v ? vd : kd, codes, scale);
      store(u.first, codes, scale);
      quantise16(r1, is_v ? vd : kd, codes, scale);
      store(u.second, codes, scale);
    }
  }
}

template <typename S, bool E4M3>
static cudaError_t launch_rows(const cudaLaunchConfig_t& cfg, const RotateArgs& a, bool single) {
  return single ? cudaLaunchKernelEx(&cfg, rotate_write_kernel<S, E4M3, 1>, a)
                : cudaLaunchKernelEx(&cfg, rotate_write_kernel<S, E4M3, kUnits>, a);
}

// Tokens of a group for 4-bit caches, whose blocks take one group each: the fewest rounds of
// units over all waves of `slots` blocks, a block's start counted as two.  (32 and 8 heads of
// 128: 1000 tokens 7.4 us, 8192 tokens 48.5 us; as many tokens as fill 768 units, one of them,
// take 8.5 and 58.3.)
static int64_t e2m1_group(int64_t tokens, int64_t all, int64_t slots) {
  int64_t best = 1, least = INT64_MAX;
  for (int64_t g = 1; g <= kMaxGroup; ++g) {
    const int64_t waves = ((tokens + g - 1) / g + slots - 1) / slots;
    const int64_t cost = waves * ((g * all + kThreads - 1) / kThreads + 2);
    if (cost < least) best = g, least = cost;
  }
  return best;
}

cudaError_t launch_rotate_write(RotateArgs a, ElemType cache, bool bf16, int num_sms,
                                cudaStream_t stream) {
  // Tokens of a group: as many as fill a block's threads with kUnits units each.  A batch
  // that so would not give every SM two blocks is latency-bound: one unit a thread, its
  // groups of one token (64 tokens of 32 and 8 heads: 3.3 us).
  const bool e2m1 = cache == ElemType::kE2m1;
  const int chunk = bf16 ? 16 : 8;               // elements of a unit
  const int64_t all = static_cast<int64_t>(a.hq) * a.dim / chunk +
                      static_cast<int64_t>(a.hk) * a.dim / (e2m1 ? 2 * kQuant : chunk) +
                      static_cast<int64_t>(a.hv) * a.v_dim / (e2m1 ? 2 * kQuant : chunk);
  if (all > (1 << 24)) return cudaErrorInvalidConfiguration;
  const int64_t full = kThreads * kUnits;
  const bool single = a.num_tokens * all < 2 * num_sms * full;
  int64_t group = single ? 1 : full / all;
  const int64_t angle_bytes = 2 * angles_of(a.rotary) * static_cast<int64_t>(sizeof(float2));
  if (e2m1) group = e2m1_group(a.num_tokens, all, 2 * num_sms);
  group = std::min(std::min<int64_t>(group, kMaxGroup), 49152 / angle_bytes);
  group = std::max<int64_t>(group, 1);
  const int64_t groups = (a.num_tokens + group - 1) / group;
  const int64_t per_block = e2m1 || single ? kThreads : kThreads * kUnits;
  int64_t parts = (group * all + per_block - 1) / per_block;
  if (parts > 65535) return cudaErrorInvalidConfiguration;
  // two blocks an SM loop over the groups; with 4-bit caches a block takes one group, in
  // parts only where that leaves room
  int64_t blocks = 2 * num_sms / parts;
  if (blocks > groups || e2m1) blocks = groups;
  if (blocks < 1) blocks = 1;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (e2m1 && blocks * parts > 2 * num_sms) parts = 1;
  a.group = static_cast<int>(group);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(group * angle_bytes / (e2m1 ? 2 : 1));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (e2m1) {
    const Divisor kd{a.k_scale, 1.f / a.k_scale}, vd{a.v_scale, 1.f / a.v_scale};
    return bf16 ? cudaLaunchKernelEx(&cfg, rotate_write_e2m1_kernel<__nv_bfloat16>, a, kd, vd)
                : cudaLaunchKernelEx(&cfg, rotate_write_e2m1_kernel<float>, a, kd, vd);
  }
  if (cache == ElemType::kE4m3)
    return bf16 ? launch_rows<__nv_bfloat16, true>(cfg, a, single)
                : launch_rows<float, true>(cfg, a, single);
  return bf16 ? launch_rows<__nv_bfloat16, false>(cfg, a, single)
              : launch_rows<float, false>(cfg, a, single);
}

}  // namespace pkv
