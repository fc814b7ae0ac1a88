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
// Persistent, warp-specialised CTA (one per SM, 352 threads):
//   warp 0      TMA producer: 128 x 128 codes of A and BN x 128 of B per
//               stage, K-major with 128-byte swizzle;
//   warp 1      owns TMEM; one thread issues tcgen05.mma (M = 128, N = BN,
//               K = 32) and commits;
//   warp 2      reads the scale bytes of four K blocks at a time into shared
//               memory in the order tcgen05.cp takes and copies them to TMEM,
//               ahead of the products;
//   warps 3..10 epilogue, two per TMEM lane quarter.
// Two accumulators (2 x BN columns) let a tile's epilogue overlap the next
// tile's products; the other columns hold kSfBufs sets of scales (so BN is at
// most 240).  Scale buffer b (shared memory and TMEM) is refilled only after
// the last product of the group that used it has completed (sf_empty).
// Every wait is bounded, as in gemm_tc_kernel.
//
// Measured: 8192 x 40960 x 1536 in 534 us (1.93 PFLOP/s; 460 us in a burst
// short of the power limit), 1001 x 4160 x 4096 in 23.8 us, 64 rows of 73728 x
// 1536 weights in 25.8 us (4.8 TB/s).
#pragma once
#include "f8_ring.h"
#include "gemm_tcgen05.cuh"

namespace csa {

struct ScaleRows {
  const uint8_t* p; long long ld;   // byte of row r, K block b: p[(r >> shift) * ld + b]
  int shift;                        // 0, or 7 for weights (one byte for 128 rows)
  int rows;                         // operand rows
};

constexpr int kF8EpiWarps = 8;                      // two per TMEM lane quarter, half of the columns each
constexpr int kF8GemmThreads = 32 * (3 + kF8EpiWarps);

struct F8GemmArgs {
  TcGemmArgs g;       // M: rows of the 128-row operand, N: of the other one
  ScaleRows sa, sb;
};

// The ring holds kGroups groups of four stages (one scale group each), so that
// a block's stage within its group is a constant of the unrolled code.
template <int BN, int kGroups>
struct F8GemmCfg {
  static constexpr int kStages = 4 * kGroups;
  static constexpr int BM = kGemmRows, BK = 128;
  static constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SFB_GROUPS = (BN + 127) / 128;           // 128-row groups of B's scales
  static constexpr int SF_BYTES = 512 * (1 + SFB_GROUPS);
  static constexpr int SF_COLS = 4 * (1 + SFB_GROUPS);
  static constexpr int kSfBufs = kGroups + 1;
  static constexpr int TMEM_COLS = 2 * BN + kSfBufs * SF_COLS <= 256 ? 256 : 512;
  static_assert(2 * BN + kSfBufs * SF_COLS <= 512, "accumulators and scales share TMEM");
  static constexpr int OUT_STAGE = kF8EpiWarps * 32 * 64;   // staging: 32 rows of 64 B per epilogue warp
  static constexpr size_t SMEM =
      1024 /*align slack*/ + (size_t)kStages * STAGE_BYTES + OUT_STAGE + (size_t)kSfBufs * SF_BYTES + 256 /*barriers*/;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// The scale bytes of K blocks 4 q .. 4 q + 3 from a row's byte 4 q on, byte by
// byte (a row's ragged end, or rows that are not 4-byte aligned); 127, a scale
// of one, past the last block: the codes there are zero.
__device__ __noinline__ uint32_t scale_bytes(const uint8_t* p, int left) {
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i) w |= (uint32_t)(i < left ? __ldg(p + i) : 127) << (8 * i);
  return w;
}
// The same as one word where that is possible.  p: NULL for a row past the matrix.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* p, int q, int k_blocks, bool words) {
  if (!p) return 0x7F7F7F7Fu;
  if (words && 4 * q + 4 <= k_blocks) return __ldg(reinterpret_cast<const uint32_t*>(p) + q);
  return scale_bytes(p + 4 * q, k_blocks - 4 * q);
}
__device__ __forceinline__ const uint8_t* scale_row(const ScaleRows& s, int r) {
  return r < s.rows ? s.p + (long long)(r >> s.shift) * s.ld : nullptr;
}

// byte offset of 16-byte piece u (0..3) of row r in 64-byte rows, XOR-swizzled
__device__ __forceinline__ uint32_t r_sw64(int r, int u) { return (uint32_t)(r * 64 + ((u ^ ((r >> 1) & 3)) << 4)); }

// ---------------------------------------------------------------- epilogue
// The MMAs of a tile take half the time of a bf16 tile's, so the epilogue
// must be short: the destination is worked out once per tile, and where the
// tile's columns lie in one segment, a step is 32 columns through the warp's
// staging rows (row = lane) and out as 64-byte pieces of rows: by 16-byte
// vectors where the rows and their ends are aligned to that, by elements where
// they are not (an odd row stride, a ragged edge).  The transposed and split
// forms go down columns (F8Column); a range across segments takes the general
// store.
struct F8Dest {
  uint8_t* p;      // row 0 of this warp's 32, column 0 of its range; NULL: general store
  long long pitch; // bytes between rows
  int rows, cols;  // in range
  int f32;
  int vec;         // whole 16-byte pieces
};

// Destination of rows r0 .. r0 + 31, columns c0 .. c0 + cols - 1 (those below
// N).
__device__ __forceinline__ F8Dest f8_dest(const TcGemmArgs& g, int r0, int c0, int cols) {
  F8Dest d;
  d.p = nullptr;
  d.pitch = 0;
  d.f32 = 0;
  d.vec = 0;
  d.rows = min(32, g.M - r0);
  d.cols = min(cols, g.N - c0);
  if (g.transpose_out || g.k_split > 1 || d.cols <= 0) return d;
#pragma unroll 1
  for (int s = 0; s < g.out.nseg; ++s) {
    const OutSeg& sg = g.out.seg[s];
    if (c0 < sg.col0 || c0 + d.cols > sg.col0 + sg.ncols) continue;
    const int es = sg.f32 ? 4 : 2;
    const long long pitch = sg.ld * es;
    uint8_t* p = static_cast<uint8_t*>(sg.ptr) + (long long)r0 * pitch + (long long)(c0 - sg.col0) * es;
    d.vec = ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)pitch | (uintptr_t)(d.cols * es)) & 15) == 0;
    d.p = p;
    d.pitch = pitch;
    d.f32 = sg.f32;
  }
  return d;
}

// The staged 64 bytes of each row by elements: a store instruction writes two
// rows of 16 fp32 or one of 32 bf16, so that neighbouring lanes are
// neighbouring addresses: 8191 x 16383 x 256 in bf16 takes 165 us, 4136 with
// a thread per row (138 for 16384 columns); 8192 x 4161 x 2048 in fp32 93,
// 1055 (74 for 4160).
template <typename T>
__device__ __noinline__ void f8_store_elements(uint8_t* p, long long pitch, int rows, int n, const uint8_t* stage) {
  constexpr int kRow = 64 / (int)sizeof(T), kRows = 32 / kRow;   // elements of a row, rows per instruction
  const int lane = threadIdx.x & 31, r0 = lane / kRow, byte = (lane % kRow) * (int)sizeof(T);
  p += (long long)r0 * pitch + byte;
  if (lane % kRow >= n) rows = 0;
#pragma unroll 8
  for (int r = r0; r < 32; r += kRows) {
    if (r < rows) *reinterpret_cast<T*>(p) = *reinterpret_cast<const T*>(stage + r_sw64(r, byte >> 4) + (byte & 15));
    p += kRows * pitch;
  }
}

// 64 bytes of each of this warp's rows (32 bf16 or 16 fp32 columns; `bytes` of
// them in range) through the staging rows: eight rows per store instruction.
__device__ __forceinline__ void f8_store_rows(const F8Dest& d, int byte0, int bytes, const uint4* v, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(stage + r_sw64(lane, u)) = v[u];
  __syncwarp();
  if (!d.vec) {
    if (bytes > 0) {
      if (d.f32) f8_store_elements<float>(d.p + byte0, d.pitch, d.rows, bytes >> 2, stage);
      else f8_store_elements<uint16_t>(d.p + byte0, d.pitch, d.rows, bytes >> 1, stage);
    }
    __syncwarp();
    return;
  }
  const int r0 = lane >> 2, u = lane & 3;
  uint8_t* p = d.p + (long long)r0 * d.pitch + byte0 + 16 * u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(stage + r_sw64(r0 + 8 * i, u));
    if (r0 + 8 * i < d.rows && 16 * u < bytes) *reinterpret_cast<uint4*>(p) = x;
    p += 8 * d.pitch;
  }
  __syncwarp();
}

// Where one value per token (or per K slice's column) goes down a column: the
// transposed and split forms.  Lanes are neighbouring output columns, so a
// step j of the warp writes 64 or 128 contiguous bytes.
struct F8Column {
  uint8_t* p;       // value of accumulator column 0 of this lane's row; NULL: none
  long long pitch;  // bytes from one accumulator column to the next
  int f32;
};
__device__ __forceinline__ F8Column f8_column(const TcGemmArgs& g, int m_tiles, int r, int ks) {
  F8Column d;
  d.p = nullptr;
  d.pitch = 0;
  d.f32 = 1;
  if (r >= g.M) return d;
  if (g.k_split > 1) {   // this K slice's fp32 sum, column j of row r at part[(ks N + j) Mpad + r]
    d.pitch = (long long)m_tiles * kGemmRows * 4;
    d.p = reinterpret_cast<uint8_t*>(g.part) + (long long)ks * g.N * d.pitch + (long long)r * 4;
    return d;
  }
#pragma unroll 1
  for (int s = 0; s < g.out.nseg; ++s) {
    const OutSeg& sg = g.out.seg[s];
    if (r < sg.col0 || r >= sg.col0 + sg.ncols) continue;
    const int es = sg.f32 ? 4 : 2;
    d.p = static_cast<uint8_t*>(sg.ptr) + (long long)(r - sg.col0) * es;
    d.pitch = sg.ld * es;
    d.f32 = sg.f32;
  }
  return d;
}
__device__ __forceinline__ void f8_store_column(const F8Column& d, int c0, int n, const float* v) {
  if (!d.p) return;
  uint8_t* p = d.p + (long long)c0 * d.pitch;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j < n) {
      if (d.f32) *reinterpret_cast<float*>(p) = v[j];
      else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v[j]);
    }
    p += d.pitch;
  }
}

// The general store of rows, out of line: it is long and rarely runs.
__device__ __noinline__ void f8_store_general(const GemmOut& out, int M, int N, int r, int c0, int n, int acc_addr) {
  float v[32];
  sm100::tmem_ld_32x32b_x32(acc_addr, v);
  if (r < M) store_chunk32<__nv_bfloat16>(out, r, c0, min(N, c0 + n), v);
}

template <int BN, int kGroups>
__global__ void __launch_bounds__(kF8GemmThreads, 1)
    gemm_f8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, F8GemmArgs a) {
  using Cfg = F8GemmCfg<BN, kGroups>;
  constexpr int kStages = Cfg::kStages;
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
  const int kbs = (k_blocks + g.k_split - 1) / g.k_split;   // K blocks per work unit (split: a multiple of 4)
  const int total = m_tiles * n_tiles * g.k_split;          // work units: (tile, K slice)

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], kF8EpiWarps);
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
      struct {
        const CUtensorMap *tmA, *tmB;
        const TcGemmArgs& g;
        uint64_t *full, *empty;
        uint8_t *smA, *smB;
        volatile int* abort_flag;
        int m_tiles, n_tiles, mt, nt;
        __device__ __forceinline__ bool aborted() const { return *abort_flag != 0; }
        __device__ __forceinline__ void abort() { *abort_flag = 1; }
        __device__ __forceinline__ void tile(int t) { gemm_tile_coords(t, m_tiles, n_tiles, g.group_m, mt, nt); }
        __device__ __forceinline__ bool wait_empty(int s, uint32_t parity) { return mbar_wait(&empty[s], parity); }
        __device__ __forceinline__ void fill(int s, int kb, bool real) {
          if (!real) {
            mbar_arrive(&full[s]);
            return;
          }
          mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
          tma_load_2d(tmA, &full[s], smA + s * Cfg::A_BYTES, kb * Cfg::BK, mt * Cfg::BM);
          tma_load_2d(tmB, &full[s], smB + s * Cfg::B_BYTES, kb * Cfg::BK, nt * BN);
        }
        __device__ __forceinline__ void wait_full(int s, uint32_t parity) { mbar_wait_small(smem_u32(&full[s]), parity); }
      } ops{&tmA, &tmB, g, full, empty, smA, smB, abort_flag, m_tiles, n_tiles, 0, 0};
      f8_fill_ring<kGroups>(ops, (int)blockIdx.x, total, (int)gridDim.x, g.k_split, kbs, k_blocks);
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ---------------- MMA issuer
      // One thread's instructions set the pace: an MMA takes BN / 2 cycles of
      // the tensor pipe, and four of them with a wait, a commit and the ring's
      // bookkeeping took this thread 480 cycles and a group's copies of scales
      // another 420.  So the scale warp copies the scales, a group of four K
      // blocks is unrolled over constant stages and constant places of the
      // scale bytes (418 cycles a block), only the descriptors' low words
      // change, and barriers are looked at ahead of the MMAs before them.
      constexpr uint32_t idesc = idesc_mxe4m3(Cfg::BM, BN, 0);
      const uint32_t a_lo0 = sdesc_lo(smem_u32(smA), 16), b_lo0 = sdesc_lo(smem_u32(smB), 16);
      const uint32_t full0 = smem_u32(full), sf_full0 = smem_u32(sf_full);
      int grp = 0, acc = 0, sb = 0;
      uint32_t phase = 0, acc_phase = 0, sf_phase = 0;
      bool ok = true;
      for (int unit = blockIdx.x; unit < total && ok && !*abort_flag; unit += gridDim.x) {
        const int kb0 = g.k_split == 1 ? 0 : (unit % g.k_split) * kbs, kb1 = min(k_blocks, kb0 + kbs);
        if (!mbar_wait_small(smem_u32(&tempty[acc]), acc_phase ^ 1)) { ok = false; break; }
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * BN);
        for (int kb = kb0; ok && kb < kb1; kb += 4) {
          const uint32_t sf_tmem = tmem_base + (uint32_t)(2 * BN + sb * Cfg::SF_COLS);
          const uint32_t full_g = full0 + 32u * (uint32_t)grp;
          const uint32_t a_lo = a_lo0 + (uint32_t)(grp * (4 * Cfg::A_BYTES >> 4)),
                         b_lo = b_lo0 + (uint32_t)(grp * (4 * Cfg::B_BYTES >> 4));
          uint32_t ready = mbar_test(full_g, phase);
          if (!mbar_wait_small(sf_full0 + 8u * (uint32_t)sb, sf_phase)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!ready && !mbar_wait_small(full_g + 8u * i, phase)) ok = false;
            if (i < 3) ready = mbar_test(full_g + 8u * (i + 1), phase);
            if (ok && kb + i < kb1) {
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < Cfg::BK / 32; ++k)
                mma_mxf8(d_tmem, a_lo + (uint32_t)(i * (Cfg::A_BYTES >> 4) + 2 * k),
                         b_lo + (uint32_t)(i * (Cfg::B_BYTES >> 4) + 2 * k), sdesc_hi(1024),
                         idesc | ((uint32_t)i << 4) | ((uint32_t)i << 29), (kb != kb0 || i != 0 || k != 0) ? 1u : 0u,
                         sf_tmem, sf_tmem + 4u);
            }
            mma_commit(&empty[4 * grp + i]);
          }
          mma_commit(&sf_empty[sb]);
          if (++sb == Cfg::kSfBufs) { sb = 0; sf_phase ^= 1; }
          if (++grp == kGroups) { grp = 0; phase ^= 1; }
        }
        mma_commit(&tfull[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
      if (!ok) *abort_flag = 1;
    }
  } else if (warp >= 3) {  // ---------------- epilogue warps 3..10
    const int sub = warp & 3;                  // TMEM lane quarter this warp may access
    const int e = warp - 3;
    constexpr int kHalf = (BN / 2 + 31) / 32 * 32;   // columns of the first four warps; the others take the rest
    const int col0 = (e >> 2) * kHalf, cols = e < 4 ? kHalf : BN - kHalf;
    const bool by_column = g.transpose_out || g.k_split > 1;
    uint8_t* stage_out = smOut + e * (32 * 64);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int unit = blockIdx.x; unit < total && !*abort_flag; unit += gridDim.x) {
      const int tile = unit / g.k_split, ks = unit % g.k_split;
      int mt, nt;
      gemm_tile_coords(tile, m_tiles, n_tiles, g.group_m, mt, nt);
      const int c0 = nt * BN + col0;
      const F8Dest d = f8_dest(g, mt * Cfg::BM + 32 * sub, c0, cols);
      F8Column fc;
      if (by_column) fc = f8_column(g, m_tiles, mt * Cfg::BM + 32 * sub + lane, ks);
      if (!mbar_wait(&tfull[acc], acc_phase)) { *abort_flag = 1; break; }
      tc_fence_after();
      __syncwarp();
      const uint32_t ta = tmem_base + ((uint32_t)(sub * 32) << 16) + (uint32_t)(acc * BN + col0);
#pragma unroll 1
      for (int c = 0; c < d.cols; c += 32) {   // (a last half step reads 16 columns too many, all of them allocated)
        if (!d.p && !by_column) {
          f8_store_general(g.out, g.M, g.N, mt * Cfg::BM + 32 * sub + lane, c0 + c, d.cols - c, (int)(ta + c));
          continue;
        }
        float v[32];
        tmem_ld_32x32b_x32(ta + (uint32_t)c, v);
        if (by_column) {
          f8_store_column(fc, c0 + c, d.cols - c, v);
        } else if (d.f32) {
          f8_store_rows(d, 4 * c, 4 * (d.cols - c), reinterpret_cast<const uint4*>(v), stage_out);
          f8_store_rows(d, 4 * c + 64, 4 * (d.cols - c) - 64, reinterpret_cast<const uint4*>(v + 16), stage_out);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          f8_store_rows(d, 2 * c, 2 * (d.cols - c), reinterpret_cast<const uint4*>(w), stage_out);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
  } else {  // ---------------- scale loader (warp 2)
    const bool words_a = ((reinterpret_cast<uintptr_t>(a.sa.p) | (uintptr_t)a.sa.ld) & 3) == 0;
    const bool words_b = ((reinterpret_cast<uintptr_t>(a.sb.p) | (uintptr_t)a.sb.ld) & 3) == 0;
    int sb = 0;
    uint32_t sf_phase = 0;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const int tile = unit / g.k_split, kb0 = (unit % g.k_split) * kbs, kb1 = min(k_blocks, kb0 + kbs);
      int mt, nt;
      gemm_tile_coords(tile, m_tiles, n_tiles, g.group_m, mt, nt);
      const uint8_t *ra[4], *rb[4 * Cfg::SFB_GROUPS];   // scale rows of this lane's operand rows
#pragma unroll
      for (int j = 0; j < 4; ++j) ra[j] = scale_row(a.sa, mt * Cfg::BM + 32 * j + lane);
#pragma unroll
      for (int j = 0; j < 4 * Cfg::SFB_GROUPS; ++j)
        rb[j] = 32 * j < BN ? scale_row(a.sb, nt * BN + 32 * j + lane) : nullptr;
      bool ok = true;
      for (int q = kb0 >> 2; 4 * q < kb1; ++q) {
        uint32_t wa[4], wb[4 * Cfg::SFB_GROUPS];
#pragma unroll
        for (int j = 0; j < 4; ++j) wa[j] = scale_word(ra[j], q, k_blocks, words_a);
#pragma unroll
        for (int j = 0; j < 4 * Cfg::SFB_GROUPS; ++j) wb[j] = scale_word(rb[j], q, k_blocks, words_b);
        if (!warp_wait_small(&sf_empty[sb], sf_phase ^ 1)) { ok = false; break; }
        uint4* dst = reinterpret_cast<uint4*>(smSf + sb * Cfg::SF_BYTES) + lane;
        dst[0] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
#pragma unroll
        for (int j = 0; j < Cfg::SFB_GROUPS; ++j)
          dst[32 * (1 + j)] = make_uint4(wb[4 * j], wb[4 * j + 1], wb[4 * j + 2], wb[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {   // to TMEM; sf_full completes with the copies
          tc_fence_after();
          const uint32_t sf_tmem = tmem_base + (uint32_t)(2 * BN + sb * Cfg::SF_COLS);
          const uint32_t sf_smem = smem_u32(smSf + sb * Cfg::SF_BYTES);
#pragma unroll
          for (int i = 0; i < 1 + Cfg::SFB_GROUPS; ++i) tmem_cp_scales(sf_tmem + 4u * (uint32_t)i, sf_smem + 512u * i);
          mma_commit(&sf_full[sb]);
        }
        __syncwarp();
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
