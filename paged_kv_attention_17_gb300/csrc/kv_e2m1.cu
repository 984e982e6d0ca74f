// Slot-mapped write into a 4-bit E2M1 cache, and the read of cached rows.
//
// "Model execution", section "Flattening a step": slot_mapping names, per new
// token, the physical slot block_id * block_size + offset of its K and V;
// section "Where it breaks": quantised KV caches are a backend feature.
//
// Write.  With t the tensor's scale, a row's 16 consecutive elements x become
//   y = RN32(x / t),  a = max |y|,
//   s = E4M3(RN32(a / 6))            (nearest even, at most 448),
//   code = E2M1(RN32(y / s))         (nearest even, at most 6; 0 if s = 0).
// a / 6 puts the block's largest element on the largest code, up to s's
// rounding.  A block holding a NaN gets the NaN scale, so the NaN is not lost.
// Bytes per token: 2 tensors x H x D x (input size + 9 / 16).  A thread takes a
// block of one tensor, the next one's inputs loaded ahead.  8192 tokens of 8 heads
// of 128 in bf16 take 12.0 us (43.1 MB, 3.6 TB/s, 53% of the measured copy
// rate); the same loads and stores without the quantising take 8.8, so latency
// and the arithmetic (eight packed fp32 operations a pair of elements for the two
// quotients) bound it, not HBM.  With plain divisions it took 18.7 us, with the
// quotients one at a time 12.8.
//
// Read.  The inverse: RN32(t * (s * code)), s * code exact, then rounded to the
// output type.  Bytes per row: 2 tensors x H x D x (9 / 16 + output size).  A
// thread takes 16 bytes of output of both tensors, striding over the rows: 64
// contexts (144 thousand rows) of 8 heads of 128 to bf16 take 119.0 us (734 MB,
// 6.17 TB/s, 91% of the measured copy rate), bound by HBM; a thread per 16 bytes
// of one tensor without the stride took 211 us.
#include "e2m1.cuh"

namespace pkv {

// One thread quantises one scale block of a token's K row, or of its V row, with
// its next block's inputs on their way.  Index is the type of the flat unit index:
// 32 bits where they hold it (its divisions are the address arithmetic).
template <typename S, int D, typename Index>
__global__ void __launch_bounds__(256, sizeof(S) == 2 ? 4 : 3) kv_write_e2m1_kernel(
    const S* __restrict__ k_new, const S* __restrict__ v_new, const int64_t* __restrict__ slots,
    Index units, uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, int64_t num_slots,
    int hkv, Divisor k_scale, Divisor v_scale, int32_t* flag) {
  using P = E2m1Page<D>;
  pdl_launch_dependents();
  pdl_wait_primary();
  const Index stride = static_cast<Index>(gridDim.x) * 256;
  Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x;   // K's units, then V's
  Raw16<S> raw;
  int64_t slot = -1;
  auto fetch = [&](Index u) {
    const bool is_v = u >= units;
    if (is_v) u -= units;
    slot = __ldg(slots + u / P::kRowScales / hkv);
    raw.load((is_v ? v_new : k_new) + static_cast<int64_t>(u) * kQuant);
  };
  if (i < 2 * units) fetch(i);
  for (; i < 2 * units; i += stride) {
    const Raw16<S> now = raw;
    const int64_t to = slot;
    if (i + stride < 2 * units) fetch(i + stride);
    const bool is_v = i >= units;
    const Index u = is_v ? i - units : i;
    const int b = static_cast<int>(u % P::kRowScales);
    const int h = static_cast<int>(u / P::kRowScales % hkv);
    if (to < 0) continue;                   // padding token: nothing to write
    if (to >= num_slots) {                  // outside the cache: skip, report
      if (b == 0 && h == 0) raise_flag(flag, PKV_FLAG_BAD_SLOT);
      continue;
    }
    uint2 codes;
    uint32_t scale;
    quantise16(now, is_v ? v_scale : k_scale, codes, scale);
    const int row = static_cast<int>(to % kBlock);
    uint8_t* page = (is_v ? v_cache : k_cache) + ((to / kBlock) * hkv + h) * P::kBytes;
    *reinterpret_cast<uint2*>(page + row * P::kRowCodes + b * (kQuant / 2)) = codes;
    page[P::kCodes + row * P::kRowScales + b] = static_cast<uint8_t>(scale);
  }
}

// One thread widens 16 bytes of output (8 bf16 or 4 fp32 elements) of a K row and
// the same of its V row, so a warp's stores are contiguous.  Index as above.
template <typename O, int D, typename Index>
__global__ void __launch_bounds__(256) kv_read_e2m1_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const int64_t* __restrict__ slots, Index units, O* __restrict__ k_out, O* __restrict__ v_out,
    int64_t num_slots, int hkv, float k_scale, float v_scale, int32_t* flag) {
  using P = E2m1Page<D>;
  constexpr int kPer = 16 / static_cast<int>(sizeof(O));
  constexpr int kRow = D / kPer;                         // units of a (row, head)
  pdl_launch_dependents();
  pdl_wait_primary();
  const Index stride = static_cast<Index>(gridDim.x) * 256;
  for (Index i = static_cast<Index>(blockIdx.x) * 256 + threadIdx.x; i < units; i += stride) {
    const int c = static_cast<int>(i % kRow);
    const Index th = i / kRow;
    const int h = static_cast<int>(th % hkv);
    const int64_t slot = __ldg(slots + th / hkv);
    if (slot < 0) continue;                 // padding row: left as it is
    if (slot >= num_slots) {
      if (c == 0 && h == 0) raise_flag(flag, PKV_FLAG_BAD_SLOT);
      continue;
    }
    const int row = static_cast<int>(slot % kBlock);
    const int64_t page = ((slot / kBlock) * hkv + h) * P::kBytes;
    const int64_t at = page + row * P::kRowCodes + c * (kPer / 2);
    const int64_t sat = page + P::kCodes + row * P::kRowScales + c * kPer / kQuant;
    auto widen = [&](const uint8_t* cache, float t, O* out) {
      uint32_t w;
      if constexpr (kPer == 8) w = __ldg(reinterpret_cast<const uint32_t*>(cache + at));
      else w = __ldg(reinterpret_cast<const uint16_t*>(cache + at));
      const float s = e4m3x2_to_float2(__ldg(cache + sat)).x;
      uint32_t r[4];
      e2m1x8_to_f16x2x4(w, r);
      float f[kPer];
#pragma unroll
      for (int k = 0; k < kPer / 2; ++k) {
        const __half2 h2 = *reinterpret_cast<const __half2*>(&r[k]);
        f[2 * k] = __low2float(h2) * s * t;             // (s * code exact: one rounding)
        f[2 * k + 1] = __high2float(h2) * s * t;
      }
      uint4 o;
      if constexpr (kPer == 8) {
        __nv_bfloat162 p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        o = *reinterpret_cast<const uint4*>(p);
      } else {
        o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
      }
      __stcs(reinterpret_cast<uint4*>(out + static_cast<int64_t>(i) * kPer), o);
    };
    widen(k_cache, k_scale, k_out);
    widen(v_cache, v_scale, v_out);
  }
}

// `per_sm` resident CTAs an SM at most, striding over the units.
static cudaLaunchConfig_t unit_config(int64_t units, int num_sms, int per_sm, cudaStream_t stream,
                                      cudaLaunchAttribute* attr) {
  const int64_t blocks = (units + 255) / 256, cap = static_cast<int64_t>(num_sms) * per_sm;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}
// (with room for a stride past the end: at most 2^21 threads)
static bool fits_32(int64_t units) { return units < (int64_t{1} << 31); }

template <typename S, int D>
static cudaError_t launch_write_t(const void* k_new, const void* v_new, const int64_t* slots,
                                  int64_t num_tokens, void* k_cache, void* v_cache,
                                  int64_t num_slots, int hkv, float k_scale, float v_scale,
                                  int32_t* flag, int num_sms, cudaStream_t stream) {
  const int64_t units = num_tokens * hkv * E2m1Page<D>::kRowScales;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      unit_config(2 * units, num_sms, sizeof(S) == 2 ? 4 : 3, stream, attr);
  auto go = [&](auto index) {
    using Index = decltype(index);
    return cudaLaunchKernelEx(&cfg, kv_write_e2m1_kernel<S, D, Index>,
                              static_cast<const S*>(k_new), static_cast<const S*>(v_new), slots,
                              static_cast<Index>(units), static_cast<uint8_t*>(k_cache),
                              static_cast<uint8_t*>(v_cache), num_slots, hkv,
                              Divisor{k_scale, 1.f / k_scale}, Divisor{v_scale, 1.f / v_scale},
                              flag);
  };
  return fits_32(2 * units) ? go(uint32_t{0}) : go(uint64_t{0});
}

cudaError_t launch_kv_write_e2m1(const void* k_new, const void* v_new, bool src_bf16,
                                 const int64_t* slots, int64_t num_tokens, void* k_cache,
                                 void* v_cache, int64_t num_slots, int hkv, int head_dim,
                                 float k_scale, float v_scale, int32_t* flag, int num_sms,
                                 cudaStream_t stream) {
  auto* f = head_dim == 128 ? (src_bf16 ? launch_write_t<__nv_bfloat16, 128>
                                        : launch_write_t<float, 128>)
                            : (src_bf16 ? launch_write_t<__nv_bfloat16, 64>
                                        : launch_write_t<float, 64>);
  return f(k_new, v_new, slots, num_tokens, k_cache, v_cache, num_slots, hkv, k_scale, v_scale,
           flag, num_sms, stream);
}

template <typename O, int D>
static cudaError_t launch_read_t(const void* k_cache, const void* v_cache, const int64_t* slots,
                                 int64_t num_rows, void* k_out, void* v_out, int64_t num_slots,
                                 int hkv, float k_scale, float v_scale, int32_t* flag, int num_sms,
                                 cudaStream_t stream) {
  const int64_t units = num_rows * hkv * (D / (16 / static_cast<int>(sizeof(O))));
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = unit_config(units, num_sms, 8, stream, attr);
  auto go = [&](auto index) {
    using Index = decltype(index);
    return cudaLaunchKernelEx(&cfg, kv_read_e2m1_kernel<O, D, Index>,
                              static_cast<const uint8_t*>(k_cache),
                              static_cast<const uint8_t*>(v_cache), slots,
                              static_cast<Index>(units), static_cast<O*>(k_out),
                              static_cast<O*>(v_out), num_slots, hkv, k_scale, v_scale, flag);
  };
  return fits_32(units) ? go(uint32_t{0}) : go(uint64_t{0});
}

cudaError_t launch_kv_read_e2m1(const void* k_cache, const void* v_cache, const int64_t* slots,
                                int64_t num_rows, void* k_out, void* v_out, bool out_bf16,
                                int64_t num_slots, int hkv, int head_dim, float k_scale,
                                float v_scale, int32_t* flag, int num_sms, cudaStream_t stream) {
  auto* f = head_dim == 128 ? (out_bf16 ? launch_read_t<__nv_bfloat16, 128>
                                        : launch_read_t<float, 128>)
                            : (out_bf16 ? launch_read_t<__nv_bfloat16, 64>
                                        : launch_read_t<float, 64>);
  return f(k_cache, v_cache, slots, num_rows, k_out, v_out, num_slots, hkv, k_scale, v_scale,
           flag, num_sms, stream);
}

}  // namespace pkv
