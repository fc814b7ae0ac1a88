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
// All kernels are one pass over HBM: a lane holds 16-byte vectors of values
// (8 bf16 or 4 fp32) in registers between the maximum and the conversion, so
// each value is read once, and the lanes of a warp take neighbouring vectors,
// so that every load and store instruction covers whole 128-byte lines.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"

namespace csa {
namespace f8 {

constexpr int kUnit = 16;    // row widths are multiples of this
constexpr int kBlock = 128;  // values per scale of a blocked row
constexpr int kSteps = 4;    // warp steps (32 vectors each) that a thread keeps in flight

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

constexpr uint32_t kInfBits = 0x7F800000u;

// Packed fp32 pairs (one instruction for two values).
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 upk2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two E4M3 codes (low and high byte of v) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// Four fp32 values to E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float2 x, float2 y) {
  uint32_t w;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(w)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return w;
}

// One 16-byte vector of a row's values.
template <typename T> struct Vec {
  static constexpr int V = Vec16<T>::V;
  uint4 v;
  __device__ __forceinline__ float at(int e) const {
    if constexpr (V == 4) return __uint_as_float(reinterpret_cast<const uint32_t*>(&v)[e]);
    const uint32_t w = reinterpret_cast<const uint32_t*>(&v)[e >> 1];
    return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);   // a bf16 is the upper half of its fp32
  }
  // fp32 bits of the largest magnitude, NaN values aside
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (V == 8) {
      __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) m = __hmax2(m, __habs2(reinterpret_cast<const __nv_bfloat162*>(&v)[q]));
      const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
      return max(w << 16, w & 0xFFFF0000u);
    }
    return __float_as_uint(fmaxf(fmaxf(fabsf(at(0)), fabsf(at(1))), fmaxf(fabsf(at(2)), fabsf(at(V - 1)))));
  }
  // the same, infinite values aside too (for blocks that hold one)
  __device__ __forceinline__ uint32_t amax_finite() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t b = __float_as_uint(at(e)) & 0x7FFFFFFFu;
      m = max(m, b < 0x7F800000u ? b : 0u);
    }
    return m;
  }
  // its V codes, to a V-byte aligned address.  kInf: the block holds infinite
  // values, which become NaN codes (a NaN value converts to one by itself).
  template <bool kInf>
  __device__ __forceinline__ void encode_to(uint8_t* dst, float inv) const {
    uint32_t w[V / 4];
    const uint64_t inv2 = pk2(inv, inv);
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      float2 x = upk2(mul2(pk2(at(4 * q), at(4 * q + 1)), inv2)), y = upk2(mul2(pk2(at(4 * q + 2), at(4 * q + 3)), inv2));
      if constexpr (kInf) {
        x.x = fabsf(x.x) < INFINITY ? x.x : NAN;
        x.y = fabsf(x.y) < INFINITY ? x.y : NAN;
        y.x = fabsf(y.x) < INFINITY ? y.x : NAN;
        y.y = fabsf(y.y) < INFINITY ? y.y : NAN;
      }
      w[q] = f32x4_to_e4m3(x, y);
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
};

// How warps walk over rows of `per` steps (32 vectors each): a warp's kSteps
// steps are kSteps neighbours in one row where rows are long enough, else the
// same step of kSteps rows, so that each is the last one plus a constant.
// Work is numbered warp by warp, `cols` warps to a row (or group of rows).
struct Walk {
  int cols, row_step, col_step;   // col_step in steps
  unsigned warps;
  int n;                          // rows
};

struct QuantArgs {
  const void* X; long long ld;            // [n, w] values
  const int* slots; int n_slots;          // destination row of row r (NULL: r); -1: not stored
  uint8_t* codes; long long ld_codes;
  uint8_t* scales; long long ld_scales;
  int n, w;
  Walk walk;
};

// The destination row of source row `row`, given its slot (loaded ahead; the
// row itself where there are no slots); -1: not stored.
__device__ __forceinline__ int load_slot(const QuantArgs& a, int row) { return a.slots ? __ldg(a.slots + row) : row; }
__device__ __forceinline__ long long quant_slot(const QuantArgs& a, int slot, bool teller) {
  if (slot >= 0 && (!a.slots || slot < a.n_slots)) return slot;
  if (slot != -1 && teller) flag_status(kStatusBadIndex);
  return -1;
}

// Row and column (of this lane) of a warp's first step; false: no such warp.
template <int V>
__device__ __forceinline__ bool walk_start(const Walk& w, int& row, int& col) {
  const unsigned i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= w.warps) return false;
  const unsigned r = i / (unsigned)w.cols, c = i - r * (unsigned)w.cols;
  row = (int)r * (w.row_step ? kSteps : 1);
  col = ((int)c * (w.row_step ? 1 : kSteps) * 32 + (int)(threadIdx.x & 31)) * V;
  return true;
}

// Blocks of 128: a warp step is 32 vectors of a row (two blocks of bf16, one
// of fp32), so that a block never crosses a step; a warp takes kSteps steps.
// Bound by issue slots before HBM when each step looked up its own row (147
// instructions a step, 23.9 us for 8192 x 4096 bf16 against 15.4 us of
// traffic); hence the constant strides, the packed arithmetic and a path of its
// own for infinite values (20.7 us, 4.9 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(QuantArgs a) {
  constexpr int V = Vec<T>::V, kStep = 32 * V;
  pdl_prologue_done();
  int row0, col0;
  if (!walk_start<V>(a.walk, row0, col0)) return;
  const int dr = a.walk.row_step, dc = a.walk.col_step * kStep;
  const T* src = static_cast<const T*>(a.X) + (long long)row0 * a.ld + col0;
  const long long ds = dr * a.ld + dc;
  Vec<T> x[kSteps];
  int slot[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    x[k].v = make_uint4(0, 0, 0, 0);
    slot[k] = -1;
    if (row0 + k * dr < a.walk.n && col0 + k * dc < a.w) {
      x[k].v = __ldcs(reinterpret_cast<const uint4*>(src + k * ds));
      slot[k] = load_slot(a, row0 + k * dr);
    }
  }
  // A step's codes and scales; kInf as for encode_to (rare, and then for the whole warp).
  auto store = [&](auto inf, int k, uint32_t m) {
    constexpr bool kInf = decltype(inf)::value;
    if constexpr (kInf) {
      m = x[k].amax_finite();
#pragma unroll
      for (int off = kBlock / V / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    }
    const int col = col0 + k * dc;
    const long long dst = quant_slot(a, slot[k], col == 0);
    if (dst < 0) return;
    const int b = scale_byte(m);
    x[k].template encode_to<kInf>(a.codes + dst * a.ld_codes + col, inv_scale(b));
    if ((col & (kBlock - 1)) == 0) a.scales[dst * a.ld_scales + (col >> 7)] = (uint8_t)b;
  };
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    uint32_t m = x[k].amax();
#pragma unroll
    for (int off = kBlock / V / 2; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (__any_sync(0xffffffffu, m >= kInfBits)) store(std::true_type{}, k, m);
    else store(std::false_type{}, k, m);
  }
}

// One scale for the whole row: one warp per row (32768 rows of 512 bf16 to
// scattered slots: 10.5 us, 4.8 TB/s).  Rows of up to kSteps steps
// (1024 bf16, 512 fp32 values) stay in registers; longer ones are read twice
// (the second time from L2).
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  constexpr int V = Vec<T>::V, kStep = 32 * V;
  pdl_prologue_done();
  const int lane = threadIdx.x & 31;
  const long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (r >= a.n) return;
  const int row = (int)r;
  const T* src = static_cast<const T*>(a.X) + (long long)row * a.ld + V * lane;
  Vec<T> x[kSteps];
  const int slot = load_slot(a, row);
  auto row_max = [&](bool finite) {
    uint32_t m = 0;
    for (int c0 = 0; c0 < a.w; c0 += kSteps * kStep) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        x[k].v = make_uint4(0, 0, 0, 0);
        if (c0 + k * kStep + V * lane < a.w) x[k].v = __ldcs(reinterpret_cast<const uint4*>(src + c0 + k * kStep));
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k) m = max(m, finite ? x[k].amax_finite() : x[k].amax());
    }
    return __reduce_max_sync(0xffffffffu, m);
  };
  uint32_t m = row_max(false);
  const bool inf = m >= kInfBits;
  if (inf) m = row_max(true);
  const long long dst = quant_slot(a, slot, lane == 0);
  if (dst < 0) return;
  const int b = scale_byte(m);
  const float inv = inv_scale(b);
  uint8_t* out = a.codes + dst * a.ld_codes + V * lane;
  const bool kept = a.w <= kSteps * kStep;
  auto store = [&](auto inf) {
    for (int c0 = 0; c0 < a.w; c0 += kSteps * kStep) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if (c0 + k * kStep + V * lane >= a.w) continue;
        if (!kept) x[k].v = __ldcs(reinterpret_cast<const uint4*>(src + c0 + k * kStep));
        x[k].template encode_to<decltype(inf)::value>(out + c0 + k * kStep, inv);
      }
    }
  };
  if (inf) store(std::true_type{});
  else store(std::false_type{});
  if (lane == 0) a.scales[dst * a.ld_scales] = (uint8_t)b;
}

// A matrix [N, K] with one scale for each 128 x 128 values: one CTA per
// square, a warp 16 of its rows (32 of a square's columns at a time per
// 128-byte line of codes).  73728 x 1536 bf16: 55 us, 6.2 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) quantize_squares_kernel(const T* W, long long ld, int N, int K, uint8_t* codes,
                                                               long long ld_codes, uint8_t* scales,
                                                               long long ld_scales) {
  constexpr int V = Vec<T>::V, kLanes = kBlock / V, kRows = 256 / kLanes, kPasses = kBlock / kRows;
  __shared__ uint32_t top[2];   // largest magnitude; largest finite one, where that is infinite
  pdl_prologue_done();
  const int k = blockIdx.x * kBlock + V * (threadIdx.x % kLanes), r0 = threadIdx.x / kLanes;
  for (int by = blockIdx.y; by * kBlock < N; by += gridDim.y) {
    if (threadIdx.x < 2) top[threadIdx.x] = 0;
    __syncthreads();
    Vec<T> x[kPasses];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = by * kBlock + r0 + kRows * i;
      x[i].v = make_uint4(0, 0, 0, 0);
      if (r < N && k < K) x[i].v = __ldcs(reinterpret_cast<const uint4*>(W + (long long)r * ld + k));
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) m = max(m, x[i].amax());
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(&top[0], m);
    __syncthreads();
    const bool inf = top[0] >= kInfBits;
    if (inf) {
      m = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) m = max(m, x[i].amax_finite());
      m = __reduce_max_sync(0xffffffffu, m);
      if ((threadIdx.x & 31) == 0) atomicMax(&top[1], m);
      __syncthreads();
    }
    const int b = scale_byte(top[inf ? 1 : 0]);
    const float inv = inv_scale(b);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = by * kBlock + r0 + kRows * i;
      if (r < N && k < K) x[i].template encode_to<true>(codes + (long long)r * ld_codes + k, inv);
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
  int w, block;                           // values of a row; per scale
  Walk walk;
};

// Read back: a warp step is 32 output vectors of a row; a warp takes kSteps.
// 131072 rows of 512 to fp32: 55.8 us, 6.0 TB/s (with a thread per 16 codes,
// whose stores covered half of each sector at a time, 73 us).
template <typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(DequantArgs a) {
  constexpr int V = Vec<T>::V, kStep = 32 * V;
  pdl_prologue_done();
  int row0, col0;
  if (!walk_start<V>(a.walk, row0, col0)) return;
  const int dr = a.walk.row_step, dc = a.walk.col_step * kStep;
  int src[kSteps];
  bool some[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int row = row0 + k * dr;
    some[k] = row < a.walk.n && col0 + k * dc < a.w;
    src[k] = row;
    if (a.rows && some[k]) {
      const int at = __ldg(a.rows + row);
      src[k] = at >= 0 && at < a.n_slots ? at : -1;
      if (src[k] < 0 && at != -1 && col0 + k * dc == 0) flag_status(kStatusBadIndex);
    }
  }
  uint32_t c[kSteps][V / 4];
  uint32_t b[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
#pragma unroll
    for (int q = 0; q < V / 4; ++q) c[k][q] = 0;
    b[k] = 127;
    if (some[k] && src[k] >= 0) {
      const int col = col0 + k * dc;
      const uint8_t* p = a.codes + src[k] * a.ld_codes + col;
      if constexpr (V == 8) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        c[k][0] = u.x;
        c[k][1] = u.y;
      } else {
        c[k][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
      b[k] = __ldg(a.scales + src[k] * a.ld_scales + (a.block == kBlock ? col >> 7 : 0));
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    if (!some[k]) continue;
    const float scale = scale_value(b[k]);
    Vec16<T> o;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 f = e4m3x2_to_f32((uint16_t)(c[k][e >> 2] >> (8 * (e & 3))));
      o.e[e] = from_f32<T>(f.x * scale);
      o.e[e + 1] = from_f32<T>(f.y * scale);
    }
    __stcs(reinterpret_cast<uint4*>(static_cast<T*>(a.X) + (long long)(row0 + k * dr) * a.ld + col0 + k * dc), o.u);
  }
}

}  // namespace f8
}  // namespace csa
