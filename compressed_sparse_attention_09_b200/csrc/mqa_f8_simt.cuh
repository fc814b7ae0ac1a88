// Shared-KV MQA over 8-bit entries (eqs. 9-11 of "Compressed Sparse
// Attention", cnblogs), CUDA-core version: mqa_simt_kernel with entries read
// as E4M3 codes under one power-of-two scale (f8_rows.cuh).  An entry's scale
// multiplies its score once and its value weight once, so the codes are only
// widened.  It takes every configuration that the tensor-core kernel does not:
// fp32 queries, other widths than c = 512, heads not in groups of 64.  Simple
// rather than fast, a CTA per row whose warps read the row's entries once for
// every two heads: 64 decode rows of 512 entries take 1209 us with 64 fp32 heads
// of 512 channels, 451 with 32 bf16 heads of 128.
#pragma once
#include "f8_rows.cuh"

namespace csa {

struct MqaF8Args {
  const void* q; long long ld_q;   // [rows, nh*c]
  const uint8_t* codes;            // entries [*, c]
  const uint8_t* scales;           // [*]
  const int* idx;                  // [rows, topk]
  void* O; long long ld_O;         // [rows, nh*c]
  int topk, nh, rows;
  float scale_log2;                // log2(e) / sqrt(c)
  RowMap rm;
};

// VEC = c / 32 channels per lane, two heads per warp pass.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) mqa_f8_simt_kernel(MqaF8Args a) {
  constexpr int C = VEC * 32;
  pdl_prologue_done();
  const int row = blockIdx.x;
  long long base;
  int avail;
  row_entries(a.rm, row, base, avail);
  const int* ir = a.idx + (long long)row * a.topk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const T* qrow = static_cast<const T*>(a.q) + (long long)row * a.ld_q;
  for (int h0 = 2 * warp; h0 < a.nh; h0 += 2 * nw) {
    const int nhp = min(2, a.nh - h0);
    float qv[2][VEC], o[2][VEC], mx[2], l[2];
#pragma unroll
    for (int hp = 0; hp < 2; ++hp) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        qv[hp][e] = hp < nhp ? to_f32(qrow[(long long)(h0 + hp) * C + lane * VEC + e]) * a.scale_log2 : 0.f;
        o[hp][e] = 0.f;
      }
      mx[hp] = -INFINITY;
      l[hp] = 0.f;
    }
    for (int j = 0; j < a.topk; ++j) {
      const int s = __ldg(ir + j);
      if (s < 0 || s >= avail) {
        if (s != -1 && lane == 0 && h0 == 0) flag_status(kStatusBadIndex);
        continue;
      }
      if (!dcheck(base + s < rowmap_entries(a.rm, a.rows))) continue;
      const uint8_t* cp = a.codes + (base + s) * C + lane * VEC;
      const float scale = f8::scale_value(__ldg(a.scales + base + s));
      float cv[VEC];
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const float2 f = f8::e4m3x2_to_f32(__ldg(reinterpret_cast<const uint16_t*>(cp + e)));
        cv[e] = f.x;
        cv[e + 1] = f.y;
      }
#pragma unroll
      for (int hp = 0; hp < 2; ++hp) {
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) d = fmaf(qv[hp][e], cv[e], d);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        d *= scale;
        const float mnew = fmaxf(mx[hp], d);
        const float alpha = exp2f(mx[hp] - mnew);   // exp2(-inf) = 0 on the first entry
        const float p = exp2f(d - mnew), w = p * scale;
        l[hp] = fmaf(l[hp], alpha, p);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[hp][e] = fmaf(o[hp][e], alpha, w * cv[e]);
        mx[hp] = mnew;
      }
    }
#pragma unroll
    for (int hp = 0; hp < 2; ++hp) {
      if (hp >= nhp) continue;
      const float inv = l[hp] == 0.f ? 0.f : 1.f / l[hp];   // nothing selected: the output is zero
      T* orow = static_cast<T*>(a.O) + (long long)row * a.ld_O + (long long)(h0 + hp) * C + lane * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) orow[e] = from_f32<T>(o[hp][e] * inv);
    }
  }
}

}  // namespace csa
