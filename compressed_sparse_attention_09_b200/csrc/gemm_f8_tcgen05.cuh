// 8-bit projection product for sm_100a:  D[M, N] = A[M, K] . B[N, K]^T over
// block-scaled E4M3 rows (f8_rows.cuh), fp32 accumulation in TMEM:
//     D[i, j] = sum_b 2^(sa[i, b] + sb[j, b] - 254) sum_{k in block b} a[i, k] b[j, k]
// with one scale byte per operand row and K block of 128 (the weights repeat
// one byte for 128 rows).
//
// The scales are powers of two held as UE8M0 bytes, which is what the tensor
// core's block-scaled form takes (kind::mxf8f6f4): it multiplies each K = 32
// product by both operands' scales before it accumulates, so the sums never
// leave TMEM between K blocks and the kernel issues nothing per block but
// its MMAs.  (An fp32 scale per block would need every 128-deep partial sum
// read back, scaled and added in registers.)
//
// A 32-bit TMEM cell holds four scale bytes and the instruction descriptor
// names one of them, so the bytes of four consecutive K blocks, which are
// four consecutive bytes of a scale row, go into one cell: one copy of scales
// per 512 values of K.
//
// Persistent, warp-specialised CTA (one per SM, 224 threads):
//   warp 0      TMA producer: 128 x 128 codes of A and BN x 128 of B per
//               stage, K-major with 128-byte swizzle;
//   warp 1      owns TMEM; one thread copies scales to TMEM (tcgen05.cp),
//               issues tcgen05.mma (M = 128, N = BN, K = 32) and commits;
//   warps 2..5  epilogue (gemm_store_cols64 of gemm_tcgen05.cuh);
//   warp 6      reads the scale bytes of four K blocks at a time into shared
//               memory in the order tcgen05.cp takes, one group ahead.
// Two accumulators (2 x BN columns) let a tile's epilogue overlap the next
// tile's products; the other columns hold kSfBufs sets of scales.  Scale
// buffer b (shared memory and TMEM) is refilled only after the last product
// of the group that used it has completed (sf_empty).
// Every wait is bounded, as in gemm_tc_kernel.
#pragma once
#include "gemm_tcgen05.cuh"

namespace csa {

struct ScaleRows {
  const uint8_t* p; long long ld;   // byte of row r, K block b: p[(r / div) * ld + b]
  int div;                          // 1, or 128 for weights
  int rows;                         // operand rows
};

struct F8GemmArgs {
  TcGemmArgs g;       // M: rows of the 128-row operand, N: of the other one
  ScaleRows sa, sb;
};

template <int BN, int kStages>
struct F8GemmCfg {
  static constexpr int BM = kGemmRows, BK = 128;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SFB_GROUPS = (BN + 127) / 128;           // 128-row groups of B's scales
  static constexpr int SF_BYTES = 512 * (1 + SFB_GROUPS);
  static constexpr int SF_COLS = 4 * (1 + SFB_GROUPS);
  static constexpr int kSfBufs = 4;
  static constexpr int TMEM_COLS = 2 * BN + kSfBufs * SF_COLS <= 256 ? 256 : 512;
  static_assert(2 * BN + kSfBufs * SF_COLS <= 512, "accumulators and scales share TMEM");
  static constexpr int OUT_STAGE = 4 * 32 * 128;
  static constexpr size_t SMEM =
      1024 /*align slack*/ + (size_t)kStages * STAGE_BYTES + OUT_STAGE + (size_t)kSfBufs * SF_BYTES + 256 /*barriers*/;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// The scale bytes of K blocks 4 q .. 4 q + 3 of operand row r (127, a scale
// of one, where there is no such row or block: the codes there are zero).
__device__ __forceinline__ uint32_t scale_word(const ScaleRows& s, int r, int q, int k_blocks) {
  if (r >= s.rows) return 0x7F7F7F7Fu;
  const uint8_t* p = s.p + (long long)(r / s.div) * s.ld + 4 * q;
  if (4 * q + 4 <= k_blocks && (reinterpret_cast<uintptr_t>(p) & 3) == 0) return __ldg(reinterpret_cast<const uint32_t*>(p));
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= (uint32_t)(4 * q + i < k_blocks ? __ldg(p + i) : 127) << (8 * i);
  return w;
}

template <int BN, int kStages>
__global__ void __launch_bounds__(224, 1)
    gemm_f8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, F8GemmArgs a) {
  using Cfg = F8GemmCfg<BN, kStages>;
  using namespace sm100;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + kStages * Cfg::A_BYTES;
  uint8_t* smOut = smem + kStages * Cfg::STAGE_BYTES;
  uint8_t* smSf = smOut + Cfg::OUT_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smSf + Cfg::kSfBufs * Cfg::SF_BYTES);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* sf_full = tempty + 2;
  uint64_t* sf_empty = sf_full + Cfg::kSfBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sf_empty + Cfg::kSfBufs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const TcGemmArgs& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tiles = (g.M + Cfg::BM - 1) / Cfg::BM;
  const int n_tiles = (g.N + BN - 1) / BN;
  const int k_blocks = (g.K + Cfg::BK - 1) / Cfg::BK;
  const int kbs = (k_blocks + g.k_split - 1) / g.k_split;   // K blocks per work unit
  const int total = m_tiles * n_tiles * g.k_split;          // work units: (tile, K slice)

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 4);
    }
    for (int s = 0; s < Cfg::kSfBufs; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_prologue_done();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {  // ---------------- TMA producer
      int stage = 0;
      uint32_t phase = 0;
      for (int unit = blockIdx.x; unit < total && !*abort_flag; unit += gridDim.x) {
        const int tile = unit / g.k_split, kb0 = (unit % g.k_split) * kbs, kb1 = min(k_blocks, kb0 + kbs);
        int mt, nt;
        gemm_tile_coords(tile, m_tiles, n_tiles, g.group_m, mt, nt);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) { *abort_flag = 1; break; }
          mbar_arrive_expect_tx(&full[stage], Cfg::STAGE_BYTES);
          tma_load_2d(&tmA, &full[stage], smA + stage * Cfg::A_BYTES, kb * Cfg::BK, mt * Cfg::BM);
          tma_load_2d(&tmB, &full[stage], smB + stage * Cfg::B_BYTES, kb * Cfg::BK, nt * BN);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ---------------- MMA issuer
      constexpr uint32_t idesc = idesc_mxe4m3(Cfg::BM, BN, 0);
      int stage = 0, acc = 0, sb = 0;
      uint32_t phase = 0, acc_phase = 0, sf_phase = 0;
      for (int unit = blockIdx.x; unit < total && !*abort_flag; unit += gridDim.x) {
        const int kb0 = (unit % g.k_split) * kbs, kb1 = min(k_blocks, kb0 + kbs);
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1)) { *abort_flag = 1; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint32_t sf_tmem = tmem_base + (uint32_t)(2 * BN + sb * Cfg::SF_COLS);
          if (kb == kb0 || (kb & 3) == 0) {   // a new group of four K blocks: its scales to TMEM
            if (!mbar_wait(&sf_full[sb], sf_phase)) { *abort_flag = 1; break; }
            tc_fence_after();
            const uint32_t sf_smem = smem_u32(smSf + sb * Cfg::SF_BYTES);
#pragma unroll
            for (int i = 0; i < 1 + Cfg::SFB_GROUPS; ++i)
              tmem_cp_scales(sf_tmem + 4u * (uint32_t)i, sf_smem + 512u * (uint32_t)i);
          }
          if (!mbar_wait(&full[stage], phase)) { *abort_flag = 1; break; }
          tc_fence_after();
          const uint64_t ad = sdesc_k_sw128(smem_u32(smA + stage * Cfg::A_BYTES));
          const uint64_t bd = sdesc_k_sw128(smem_u32(smB + stage * Cfg::B_BYTES));
          const uint32_t sf_id = (uint32_t)(kb & 3);
#pragma unroll
          for (int k = 0; k < Cfg::BK / 32; ++k)
            mma_mxf8(d_tmem, desc_add(ad, k * 32), desc_add(bd, k * 32), idesc | (sf_id << 4) | (sf_id << 29),
                     (kb != kb0 || k != 0) ? 1u : 0u, sf_tmem, sf_tmem + 4u);
          mma_commit(&empty[stage]);
          if (++stage == kStages) { stage = 0; phase ^= 1; }
          if ((kb & 3) == 3 || kb == kb1 - 1) {
            mma_commit(&sf_empty[sb]);
            if (++sb == Cfg::kSfBufs) { sb = 0; sf_phase ^= 1; }
          }
        }
        mma_commit(&tfull[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
  } else if (warp < 6) {  // ---------------- epilogue warps 2..5
    const int sub = warp & 3;   // TMEM lane quarter this warp may access
    uint8_t* stage_out = smOut + (warp - 2) * (32 * 128);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int unit = blockIdx.x; unit < total && !*abort_flag; unit += gridDim.x) {
      const int tile = unit / g.k_split, ks = unit % g.k_split;
      int mt, nt;
      gemm_tile_coords(tile, m_tiles, n_tiles, g.group_m, mt, nt);
      if (!mbar_wait(&tfull[acc], acc_phase)) { *abort_flag = 1; break; }
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < BN / 64; ++ch) {
        float v0[32], v1[32];
        const uint32_t ta = tmem_base + ((uint32_t)(sub * 32) << 16) + (uint32_t)(acc * BN + ch * 64);
        tmem_ld_32x32b_x32_pair(ta, ta + 32u, v0, v1);
        gemm_store_cols64(g, m_tiles, mt, sub, ks, nt * BN + ch * 64, v0, v1, stage_out);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  } else {  // ---------------- scale loader (warp 6)
    int sb = 0;
    uint32_t sf_phase = 0;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const int tile = unit / g.k_split, kb0 = (unit % g.k_split) * kbs, kb1 = min(k_blocks, kb0 + kbs);
      int mt, nt;
      gemm_tile_coords(tile, m_tiles, n_tiles, g.group_m, mt, nt);
      bool ok = true;
      for (int q = kb0 >> 2; q <= (kb1 - 1) >> 2; ++q) {
        uint32_t wa[4], wb[4 * Cfg::SFB_GROUPS];
#pragma unroll
        for (int j = 0; j < 4; ++j) wa[j] = scale_word(a.sa, mt * Cfg::BM + 32 * j + lane, q, k_blocks);
#pragma unroll
        for (int j = 0; j < 4 * Cfg::SFB_GROUPS; ++j)
          wb[j] = 32 * j < BN ? scale_word(a.sb, nt * BN + 32 * j + lane, q, k_blocks) : 0x7F7F7F7Fu;
        if (!warp_wait(&sf_empty[sb], sf_phase ^ 1)) { ok = false; break; }
        uint4* dst = reinterpret_cast<uint4*>(smSf + sb * Cfg::SF_BYTES) + lane;
        dst[0] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
#pragma unroll
        for (int j = 0; j < Cfg::SFB_GROUPS; ++j)
          dst[32 * (1 + j)] = make_uint4(wb[4 * j], wb[4 * j + 1], wb[4 * j + 2], wb[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[sb]);
        if (++sb == Cfg::kSfBufs) { sb = 0; sf_phase ^= 1; }
      }
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace csa
