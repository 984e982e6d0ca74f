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
// Bytes per token: 2 tensors x H x D x (input size + 9 / 16).
//
// Read.  The inverse: RN32(t * (s * code)), s * code exact, then rounded to the
// output type.  Bytes per row: 2 tensors x H x D x (9 / 16 + output size).
#include "e2m1.cuh"

namespace pkv {

// One thread quantises one scale block of a token's K row and the same block
// of its V row.
template <typename S, int D>
__global__ void __launch_bounds__(256) kv_write_e2m1_kernel(
    const S* __restrict__ k_new, const S* __restrict__ v_new, const int64_t* __restrict__ slots,
    int64_t num_tokens, uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache,
    int64_t num_slots, int hkv, float k_scale, float v_scale, int32_t* flag) {
  using P = E2m1Page<D>;
  pdl_launch_dependents();
  pdl_wait_primary();
  const Divisor kd = divisor(k_scale), vd = divisor(v_scale);
  const int64_t total = num_tokens * hkv * P::kRowScales;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int b = static_cast<int>(i % P::kRowScales);
    const int64_t th = i / P::kRowScales;
    const int h = static_cast<int>(th % hkv);
    const int64_t slot = __ldg(slots + th / hkv);
    float kf[16], vf[16];
    load16(k_new + i * kQuant, kf);
    load16(v_new + i * kQuant, vf);
    if (slot < 0) continue;                 // padding token: nothing to write
    if (slot >= num_slots) {                // outside the cache: skip, report
      if (b == 0 && h == 0) raise_flag(flag, PKV_FLAG_BAD_SLOT);
      continue;
    }
    const int row = static_cast<int>(slot % kBlock);
    const int64_t page = ((slot / kBlock) * hkv + h) * P::kBytes;
    const int64_t at = page + row * P::kRowCodes + b * (kQuant / 2);
    const int64_t sat = page + P::kCodes + row * P::kRowScales + b;
    uint2 codes;
    uint32_t scale;
    quantise16(kf, kd, codes, scale);
    *reinterpret_cast<uint2*>(k_cache + at) = codes;
    k_cache[sat] = static_cast<uint8_t>(scale);
    quantise16(vf, vd, codes, scale);
    *reinterpret_cast<uint2*>(v_cache + at) = codes;
    v_cache[sat] = static_cast<uint8_t>(scale);
  }
}

// One thread widens the 16 bytes of output (8 bf16 or 4 fp32 elements) of a K
// row and the same of its V row, so a warp's stores are contiguous.
template <typename O, int D>
__global__ void __launch_bounds__(256) kv_read_e2m1_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const int64_t* __restrict__ slots, int64_t num_rows, O* __restrict__ k_out,
    O* __restrict__ v_out, int64_t num_slots, int hkv, float k_scale, float v_scale,
    int32_t* flag) {
  using P = E2m1Page<D>;
  constexpr int kPer = 16 / static_cast<int>(sizeof(O));
  constexpr int kRow = D / kPer;                         // threads per (row, head)
  pdl_launch_dependents();
  pdl_wait_primary();
  const int64_t total = num_rows * hkv * kRow;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int c = static_cast<int>(i % kRow);
    const int64_t th = i / kRow;
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
      if constexpr (kPer == 8) w = *reinterpret_cast<const uint32_t*>(cache + at);
      else w = *reinterpret_cast<const uint16_t*>(cache + at);
      const float s = e4m3x2_to_float2(cache[sat]).x;
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
      __stcs(reinterpret_cast<uint4*>(out + i * kPer), o);
    };
    widen(k_cache, k_scale, k_out);
    widen(v_cache, v_scale, v_out);
  }
}

static cudaLaunchConfig_t row_config(int64_t total, int num_sms, cudaStream_t stream,
                                     cudaLaunchAttribute* attr) {
  const int threads = 256;
  int64_t blocks = (total + threads - 1) / threads;
  const int64_t cap = static_cast<int64_t>(num_sms) * 8;
  if (blocks > cap) blocks = cap;
  if (blocks < 1) blocks = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename S, int D>
static cudaError_t launch_write_t(const void* k_new, const void* v_new, const int64_t* slots,
                                  int64_t num_tokens, void* k_cache, void* v_cache,
                                  int64_t num_slots, int hkv, float k_scale, float v_scale,
                                  int32_t* flag, int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      row_config(num_tokens * hkv * E2m1Page<D>::kRowScales, num_sms, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_write_e2m1_kernel<S, D>, static_cast<const S*>(k_new),
                            static_cast<const S*>(v_new), slots, num_tokens,
                            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                            num_slots, hkv, k_scale, v_scale, flag);
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
                                 int hkv, float k_scale, float v_scale, int32_t* flag,
                                 int num_sms, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = row_config(
      num_rows * hkv * (D / (16 / static_cast<int>(sizeof(O)))), num_sms, stream, attr);
  return cudaLaunchKernelEx(&cfg, kv_read_e2m1_kernel<O, D>,
                            static_cast<const uint8_t*>(k_cache),
                            static_cast<const uint8_t*>(v_cache), slots, num_rows,
                            static_cast<O*>(k_out), static_cast<O*>(v_out), num_slots, hkv,
                            k_scale, v_scale, flag);
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
