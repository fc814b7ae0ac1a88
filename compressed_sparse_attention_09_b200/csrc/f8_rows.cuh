// Block-scaled E4M3 rows: the 8-bit format of the cache entries and of the
// operands of the 8-bit product (a format of this implementation; the page
// fixes no precision).
//
// Format.  A row of w values is w E4M3 codes and one scale byte for each
// block of the row (128 values, or the whole row).  A code c under the scale
// byte b stands for c * 2^(b - 127).  For a block with the largest finite
// magnitude A, b is the smallest byte with A <= 448 * 2^(b - 127):
//     A = 1.f * 2^(E - 127)  =>  b = E - 8 + (1.f > 1.75), at least 0,
// read off the bits of A, and code = E4M3(x * 2^(127 - b)), to nearest even.
// A power of two costs E4M3 no precision (its steps are relative), the
// multiplication by it is exact, decoding is exact in bf16, and the tensor
// cores take the byte as it is (kind::mxf8f6f4).  An infinite or NaN value is
// stored as the NaN code and leaves the block's scale alone; a block without
// a finite non-zero value gets byte 0.
//
// All three kernels are one pass over HBM: a thread holds 16 consecutive
// values (a 16-byte store of codes) in registers between the maximum and the
// conversion, so each value is read once.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace csa {
namespace f8 {

constexpr int kUnit = 16;    // values per thread: one 16-byte store of codes
constexpr int kBlock = 128;  // values per scale of a blocked row

// Scale byte of a block whose largest finite magnitude has these fp32 bits.
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  return max((int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);
}
// 2^(127 - b), the factor from values to codes (b <= 247 here, so it is a normal number)
__device__ __forceinline__ float inv_scale(int b) { return __uint_as_float((uint32_t)(254 - b) << 23); }
// 2^(b - 127); byte 0 is the subnormal 2^-127, byte 255 is NaN
__device__ __forceinline__ float scale_value(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b << 23);
}

// Two E4M3 codes (low and high byte of v) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Two fp32 values to E4M3 codes, `lo` in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// 16 consecutive values of a row, as loaded (streamed: read once).
template <typename T> struct Unit {
  static constexpr int kVecs = kUnit / Vec16<T>::V;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void load_shared(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = *(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int e) const { return to_f32(reinterpret_cast<const T*>(v)[e]); }
  // fp32 bits of the largest finite magnitude
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < kUnit; ++e) {
      const uint32_t b = __float_as_uint(at(e)) & 0x7FFFFFFFu;
      m = max(m, b < 0x7F800000u ? b : 0u);
    }
    return m;
  }
  __device__ __forceinline__ uint4 encode(float inv) const {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = at(4 * q + e);
        x[e] = fabsf(a) < INFINITY ? a * inv : NAN;
      }
      w[q] = f32x2_to_e4m3(x[0], x[1]) | (f32x2_to_e4m3(x[2], x[3]) << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// 16 codes times one factor, as 16 values of T.
template <typename T>
__device__ __forceinline__ void decode_unit(const uint4& c, float scale, T* dst) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < kUnit / Vec16<T>::V; ++i) {
    Vec16<T> o;
#pragma unroll
    for (int e = 0; e < Vec16<T>::V; e += 2) {
      const int k = i * Vec16<T>::V + e;
      const float2 f = e4m3x2_to_f32((uint16_t)(w[k >> 2] >> (8 * (k & 3))));
      o.e[e] = from_f32<T>(f.x * scale);
      o.e[e + 1] = from_f32<T>(f.y * scale);
    }
    __stcs(reinterpret_cast<uint4*>(dst) + i, o.u);
  }
}

struct QuantArgs {
  const void* X; long long ld;            // [n, w] values
  const int* slots; int n_slots;          // destination row of row r (NULL: r); -1: not stored
  uint8_t* codes; long long ld_codes;
  uint8_t* scales; long long ld_scales;
  int n, w;
  int row0;                               // first row of this launch
};

__device__ __forceinline__ long long quant_slot(const QuantArgs& a, int row, bool teller) {
  if (!a.slots) return row;
  const int s = __ldg(a.slots + row);
  if (s >= 0 && s < a.n_slots) return s;
  if (s != -1 && teller) flag_status(kStatusBadIndex);
  return -1;
}

// Blocks of 128: eight neighbouring threads share a block.  A row takes
// 8 * ceil(w / 128) threads, so that a block never crosses a warp.
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(QuantArgs a, unsigned units) {
  pdl_prologue_done();
  const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;
  const unsigned per = 8u * (unsigned)((a.w + kBlock - 1) / kBlock);
  const unsigned r = i / per, u = i - r * per;
  const bool some = i < units && (int)(u * kUnit) < a.w;
  const int row = a.row0 + (int)r;
  Unit<T> x;
  if (some) x.load(static_cast<const T*>(a.X) + (long long)row * a.ld + u * kUnit);
  else x.clear();
  uint32_t m = x.amax();
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
  if (!some) return;
  const long long dst = quant_slot(a, row, u == 0);
  if (dst < 0) return;
  const int b = scale_byte(m);
  *reinterpret_cast<uint4*>(a.codes + dst * a.ld_codes + u * kUnit) = x.encode(inv_scale(b));
  if ((u & 7) == 0) a.scales[dst * a.ld_scales + (u >> 3)] = (uint8_t)b;
}

// One scale for the whole row: one warp per row.  Rows of up to 1024 values
// stay in registers; longer ones are read twice (the second time from L2).
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  pdl_prologue_done();
  const int lane = threadIdx.x & 31;
  const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (r >= a.n) return;
  const int row = (int)r, units = a.w / kUnit;
  const T* src = static_cast<const T*>(a.X) + (long long)row * a.ld;
  Unit<T> x[2];
  uint32_t m = 0;
  for (int u0 = 0; u0 < units; u0 += 64) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = u0 + 32 * k + lane;
      if (u < units) x[k].load(src + u * kUnit);
      else x[k].clear();
    }
    m = max(m, max(x[0].amax(), x[1].amax()));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  const long long dst = quant_slot(a, row, lane == 0);
  if (dst < 0) return;
  const int b = scale_byte(m);
  const float inv = inv_scale(b);
  for (int u0 = 0; u0 < units; u0 += 64) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int u = u0 + 32 * k + lane;
      if (u >= units) continue;
      if (units > 64) x[k].load(src + u * kUnit);
      *reinterpret_cast<uint4*>(a.codes + dst * a.ld_codes + u * kUnit) = x[k].encode(inv);
    }
  }
  if (lane == 0) a.scales[dst * a.ld_scales] = (uint8_t)b;
}

// A matrix [N, K] with one scale for each 128 x 128 values: one CTA per
// square, a thread holding 16 columns of four rows.
template <typename T>
__global__ void __launch_bounds__(256) quantize_squares_kernel(const T* W, long long ld, int N, int K, uint8_t* codes,
                                                               long long ld_codes, uint8_t* scales,
                                                               long long ld_scales) {
  __shared__ uint32_t top;
  pdl_prologue_done();
  const int k0 = blockIdx.x * kBlock, u = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  for (int by = blockIdx.y; by * kBlock < N; by += gridDim.y) {
    if (threadIdx.x == 0) top = 0;
    __syncthreads();
    Unit<T> x[4];
    uint32_t m = 0;
    const int k = k0 + u * kUnit;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = by * kBlock + r0 + 32 * i;
      if (r < N && k < K) x[i].load(W + (long long)r * ld + k);
      else x[i].clear();
      m = max(m, x[i].amax());
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(&top, m);
    __syncthreads();
    const int b = scale_byte(top);
    const float inv = inv_scale(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = by * kBlock + r0 + 32 * i;
      if (r < N && k < K) *reinterpret_cast<uint4*>(codes + (long long)r * ld_codes + k) = x[i].encode(inv);
    }
    if (threadIdx.x == 0) scales[(long long)by * ld_scales + blockIdx.x] = (uint8_t)b;
    __syncthreads();
  }
}

struct DequantArgs {
  const uint8_t* codes; long long ld_codes;
  const uint8_t* scales; long long ld_scales;
  const int* rows; int n_slots;           // source row of output row r (NULL: r); -1: zeros
  void* X; long long ld;
  int w, block_units;                     // 16-value units of a row's scale block
  int row0;
};

// Read back: one thread per 16 codes.
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(DequantArgs a, unsigned units) {
  pdl_prologue_done();
  const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= units) return;
  const unsigned per = (unsigned)(a.w / kUnit);
  const unsigned r = i / per, u = i - r * per;
  const int row = a.row0 + (int)r;
  long long src = row;
  if (a.rows) {
    const int s = __ldg(a.rows + row);
    src = s >= 0 && s < a.n_slots ? s : -1;
    if (src < 0 && s != -1 && u == 0) flag_status(kStatusBadIndex);
  }
  uint4 c = make_uint4(0, 0, 0, 0);
  float scale = 0.f;
  if (src >= 0) {
    c = __ldg(reinterpret_cast<const uint4*>(a.codes + src * a.ld_codes) + u);
    scale = scale_value(__ldg(a.scales + src * a.ld_scales + u / (unsigned)a.block_units));
  }
  decode_unit<T>(c, scale, static_cast<T*>(a.X) + (long long)row * a.ld + u * kUnit);
}

}  // namespace f8
}  // namespace csa
