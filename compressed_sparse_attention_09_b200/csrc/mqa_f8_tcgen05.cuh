// Shared-KV MQA over 8-bit entries, eqs. (9)-(11) of "Compressed Sparse
// Attention" (cnblogs), on the 8-bit tensor cores of sm_100a (c = 512, heads
// in groups of 64, bf16 queries).
//
// Both operands of both products are E4M3, so the gathered codes feed the
// tensor cores as they are: no widening pass, half the shared memory and half
// the gather of a bf16 tile.  The other operand keeps its precision by being
// split into two E4M3 parts:
//   q = 2^k (hi + lo / 32)   per head, k from the row's maximum: a bf16 value
//                            has 8 significant bits, hi takes the upper 4 and
//                            lo the rest, so the split is exact (down to
//                            2^-22 of the row's largest value);
//   w = hi + lo              the softmax weight times the entry's scale: about
//                            8 bits (its rounding error, rms 0.06 %, is below
//                            that of a bf16 weight, 0.11 %).
// A work item is one query row and 64 of its heads (and a range of its tiles
// where rows are few).  Per tile of 128 selected entries
//   S[128, 128] = [hi; lo] . C^T    M = 128 (64 heads x hi, lo), N = 128
//                                   entries, K = 512: 16 MMAs, the full rate
//                                   that 64 heads alone (M = 64) cannot reach
//   s = scale_q scale_e (S_hi + S_lo / 32), w = 2^(s + e - M) on the fly
//   O[64, 512] += w_hi . C + w_lo . C    M = 64, N = 2 x 256 channels, K = 128
// where 2^e is the entry's scale (a power of two: it moves into the exponent)
// and M the running maximum of s + e, so that the weights use E4M3's range
// whatever the entries' scales are.  The normaliser is summed in fp32 from
// the unrounded probabilities.
//
// The codes sit in shared memory once, [4 chunks of 128 channels][256 ring
// entries][128 bytes] in the 128-byte swizzle: S reads 128 entries as a
// K-major operand, O reads the same bytes MN-major (32 entries = K, 256
// channels = N, two chunks apart by the ring's length).  The ring is filled
// and released in parts of 64 entries and read by S in tiles of 128.
//
// TMEM (512 columns): O in columns 0-255 (channels 0-255 in the lower 16
// lanes of every lane quarter, 256-511 in the upper 16); two S buffers of 128
// columns.  Lane quarter `sub` holds heads 16 sub .. + 15: their hi rows in
// its lower 16 lanes, their lo rows in the upper 16.
//
// Warps (20): 0-7 gather codes (16-byte cp.async, one entry per warp and
// instruction) and convert q; 8 fetches the entries' scale bytes; 9 issues S,
// 10 issues O (one thread each), 11 owns TMEM; 12-19 softmax and epilogue.
// The two softmax warps of a lane quarter take 64 entries of a tile each and
// exchange their tile maxima through shared memory (xch).
// Every wait is bounded (sm100::mbar_wait); the pairs meet on an mbarrier,
// never on a named barrier, so a wait that ran out cannot strand a partner.
#pragma once
#include "mqa_f8_simt.cuh"
#include "mqa_tcgen05.cuh"

namespace csa {

struct MqaF8TcArgs {
  const __nv_bfloat16* q; long long ld_q;   // [rows, nh*512]
  const uint8_t* codes;                     // entries [*, 512]
  const uint8_t* scales;                    // [*]
  const int* idx;                           // [rows, topk]
  __nv_bfloat16* O; long long ld_O;         // [rows, nh*512]
  int topk, nh, rows;
  float scale_log2;                         // log2(e) / sqrt(c)
  RowMap rm;
  int splits;                               // work items per (row, head group)
  int tiles_per_split;
  float* part_o;                            // splits > 1: [rows, nh, splits, 512]
  float* part_lse;                          //             [rows, nh, splits], base 2; -inf: nothing seen
};

namespace mqaf8 {
constexpr int kC = 512, kHeads = 64, kTile = 128, kPart = 64, kParts = 4;
constexpr int kChunk = kParts * kPart * 128;      // ring bytes of one 128-channel chunk
constexpr int kQChunk = 128 * 128;                // q: 128 rows x 128 channels
constexpr int kPHalf = 64 * 128;                  // 64 heads x 128 entries
constexpr int kPBytes = 2 * kPHalf;               // hi, lo
constexpr int kOffC = 4 * kQChunk;
constexpr int kOffP = kOffC + 4 * kChunk;         // two P buffers; the epilogue's staging rows between items
constexpr int kOffE = kOffP + 2 * kPBytes;        // scale byte of each ring entry
constexpr int kOffX = kOffE + kParts * kPart;     // xch: [2][8 warps][16 heads] fp32
constexpr int kOffS = kOffX + 2 * 8 * 16 * 4;     // q scale of each head
constexpr int kOffMisc = kOffS + kHeads * 4;
constexpr size_t kSmem = 1024 + kOffMisc + 512;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr int kThreads = 640;
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;
// w <= 2^(kOff + kGrow) = 256 < 448: the running maximum may lag by kGrow
constexpr float kOff = 6.f, kGrow = 2.f;
constexpr float kLo = 32.f;                       // q: lo = 32 (q - hi) is at most 256
}  // namespace mqaf8

// Tiles of 128 slots up to the row's last valid slot (0 <= s < avail), by a
// whole warp; every warp role derives it from the index row.  The row is read
// from its end, 512 slots at a time, so a full row costs one memory latency.
__device__ __forceinline__ int mqa_f8_ntiles(const int* ir, int topk, int avail) {
  const int lane = threadIdx.x & 31;
  for (int j0 = ((topk - 1) / 512) * 512; j0 >= 0; j0 -= 512) {
    int v[16], last = -1;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int j = j0 + 32 * u + lane;
      v[u] = j < topk ? __ldg(ir + j) : -1;
    }
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (v[u] >= 0 && v[u] < avail) last = j0 + 32 * u + lane;
    last = __reduce_max_sync(0xffffffffu, last);
    if (last >= 0) return last / mqaf8::kTile + 1;
  }
  return 0;
}

// E4M3 pairs <-> fp16 pairs (hardware conversions).
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(v) : "r"(h));
  return v;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}

// 32 consecutive TMEM columns from `t0` and 32 from `t1`, 16 at a time, to
// s[k] = a * x0[k] + b * x1[k] of the lane pair (L, L ^ 16): the lower lane
// keeps columns t0 .., the upper one t1 .., each giving the other's away.
__device__ __forceinline__ void tmem_ld_x16_pair(uint32_t t0, uint32_t t1, float* v0, float* v1) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t0), "r"(t1)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v0[i] = __uint_as_float(r[i]);
    v1[i] = __uint_as_float(r[16 + i]);
  }
}

__global__ void __launch_bounds__(mqaf8::kThreads, 1) mqa_f8_tc_kernel(MqaF8TcArgs a) {
  using namespace sm100;
  using namespace mqaf8;
  constexpr uint32_t kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* e_s = sm + kOffE;
  float* xch = reinterpret_cast<float*>(sm + kOffX);
  float* qs_s = reinterpret_cast<float*>(sm + kOffS);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + kOffMisc);
  uint64_t* q_empty = q_full + 1;         // the item's last S done, and every softmax warp has its q scales
  uint64_t* c_full = q_empty + 1;         // [kParts] codes landed
  uint64_t* e_full = c_full + kParts;     // [kParts] scale bytes and validity written
  uint64_t* t_done = e_full + kParts;     // [kParts] O product of the part done (frees it)
  uint64_t* s_full = t_done + kParts;     // [2]
  uint64_t* s_free = s_full + 2;          // [2]
  uint64_t* p_full = s_free + 2;          // [2]
  uint64_t* o_free = p_full + 2;
  uint64_t* x_bar = o_free + 1;           // [4] softmax pairs
  uint32_t* valid_s = reinterpret_cast<uint32_t*>(x_bar + 4);   // [kParts][2] validity of the ring entries
  uint32_t* tmem_slot = valid_s + 2 * kParts;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hgroups = a.nh / kHeads;
  const int per_row = hgroups * a.splits;
  const int items = a.rows * per_row;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    mbar_init(q_empty, 1 + 8);
    for (int s = 0; s < kParts; ++s) {
      mbar_init(&c_full[s], 256);
      mbar_init(&e_full[s], 1);
      mbar_init(&t_done[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 8);
      mbar_init(&p_full[s], 8);
    }
    mbar_init(o_free, 8);
    for (int s = 0; s < 4; ++s) mbar_init(&x_bar[s], 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 11) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_prologue_done();
  const uint32_t tmem = *tmem_slot;

  // An item: its row and head group, and the tiles [t0, t1) of the row that
  // it covers.  Rows run last first: they see the most entries.
  struct Item {
    int row, hg, split, t0, t1, avail;
    long long base;
    const int* ir;
  };
  auto item_of = [&](int it) {
    Item w;
    w.row = a.rows - 1 - it / per_row;
    const int r = it % per_row;
    w.hg = r / a.splits;
    w.split = r - w.hg * a.splits;
    row_entries(a.rm, w.row, w.base, w.avail);
    w.ir = a.idx + (long long)w.row * a.topk;
    const int n = mqa_f8_ntiles(w.ir, a.topk, w.avail);
    w.t0 = w.split * a.tiles_per_split;
    w.t1 = min(n, w.t0 + a.tiles_per_split);
    return w;
  };

  if (warp < 8) {
    // ------------------------------------------------------------ gather and q conversion (warps 0-7)
    uint32_t g = 0, qw = 0;   // ring parts, items
    bool ok = true;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const Item w = item_of(it);
      if (w.t0 >= w.t1) continue;
      const long long n_ent = rowmap_entries(a.rm, a.rows);
      // q: this warp's heads 8 warp .. + 7, a lane 16 channels of each (four heads in flight)
      const __nv_bfloat16* qrow =
          a.q + (long long)w.row * a.ld_q + (long long)(w.hg * kHeads + 8 * warp) * kC + 16 * lane;
#pragma unroll 1
      for (int hb = 0; hb < 2; ++hb) {
        uint4 raw[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) raw[i][u] = __ldg(reinterpret_cast<const uint4*>(qrow + (4 * hb + i) * kC) + u);
        if (hb == 0 && !warp_wait(q_empty, (qw & 1) ^ 1)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t* rw = reinterpret_cast<const uint32_t*>(raw[i]);
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t x0 = (rw[e] << 16) & 0x7FFFFFFFu, x1 = rw[e] & 0x7FFF0000u;
            m = max(m, max(x0 < 0x7F800000u ? x0 : 0u, x1 < 0x7F800000u ? x1 : 0u));
          }
          m = __reduce_max_sync(kFull, m);
          // 2^-k with the largest value in [128, 256)
          const uint32_t ex = max(m >> 23, 8u);
          const float inv = __uint_as_float((261u - ex) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            hi[q] = 0;
            lo[q] = 0;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t wd = rw[2 * q + p];
              float x0 = __uint_as_float(wd << 16), x1 = __uint_as_float(wd & 0xFFFF0000u);
              x0 = fabsf(x0) < INFINITY ? x0 * inv : NAN;
              x1 = fabsf(x1) < INFINITY ? x1 * inv : NAN;
              const uint32_t h = f8::f32x2_to_e4m3(x0, x1);
              const float2 hf = f8::e4m3x2_to_f32((uint16_t)h);
              hi[q] |= h << (16 * p);
              lo[q] |= f8::f32x2_to_e4m3((x0 - hf.x) * kLo, (x1 - hf.y) * kLo) << (16 * p);
            }
          }
          const int head = 8 * warp + 4 * hb + i;
          const int r = 32 * (head >> 4) + (head & 15);
          uint8_t* dst = sm + (lane >> 3) * kQChunk;
          *reinterpret_cast<uint4*>(dst + sw128(r, lane & 7)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + sw128(r + 16, lane & 7)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (lane == 0) qs_s[head] = __uint_as_float((ex - 7u) << 23);
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      ++qw;
      // codes: entry warp + 8 i of a part per instruction, a lane 16 bytes; slots fetched one part ahead
      const int p0 = 2 * w.t0, p1 = 2 * w.t1;
      auto slot = [&](int p) {
        const int e = p * kPart + warp + 8 * lane;
        return lane < 8 && e < a.topk ? __ldg(w.ir + e) : -1;
      };
      int next = slot(p0);
      for (int p = p0; p < p1; ++p, ++g) {
        const int st = (int)(g % kParts);
        const int mine = next;
        next = p + 1 < p1 ? slot(p + 1) : -1;
        if (!warp_wait(&t_done[st], ((g / kParts) & 1) ^ 1)) { ok = false; break; }
        uint8_t* dst = sm + kOffC + (lane >> 3) * kChunk + st * kPart * 128;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = __shfl_sync(kFull, mine, i);
          const bool v = s >= 0 && s < w.avail && dcheck(w.base + s < n_ent);
          const uint8_t* src = v ? a.codes + (w.base + s) * kC + 16 * lane : a.codes;
          cp_async16(dst + sw128(warp + 8 * i, lane & 7), src, v ? 16u : 0u);
        }
        cp_async_arrive_noinc(&c_full[st]);
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    cp_async_wait_all();
  } else if (warp == 8) {
    // ------------------------------------------------------------ scale bytes and validity
    uint32_t g = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const Item w = item_of(it);
      bool ok = true;
      for (int p = 2 * w.t0; p < 2 * w.t1; ++p, ++g) {
        const int st = (int)(g % kParts);
        bool v[2];
        uint32_t b[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int e = p * kPart + 32 * u + lane;
          const int s = e < a.topk ? __ldg(w.ir + e) : -1;
          v[u] = s >= 0 && s < w.avail;
          if (!v[u] && s != -1) flag_status(kStatusBadIndex);
          b[u] = v[u] ? __ldg(a.scales + w.base + s) : 0u;
        }
        if (!warp_wait(&t_done[st], ((g / kParts) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          e_s[st * kPart + 32 * u + lane] = (uint8_t)b[u];
          const uint32_t m = __ballot_sync(kFull, v[u]);
          if (lane == 0) valid_s[2 * st + u] = m;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&e_full[st]);
      }
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ S issuer (lane 0)
    constexpr uint32_t idS = idesc_e4m3_f32(128, kTile);
    const uint64_t qd0 = sdesc_k_sw128(smem_u32(sm));
    const uint64_t cd0 = sdesc_k_sw128(smem_u32(sm + kOffC));
    uint32_t g = 0, qw = 0;   // tiles, items
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const Item w = item_of(it);
      if (w.t0 >= w.t1) continue;
      int ok = 1;
      if (lane == 0) {
        if (!mbar_wait(q_full, qw & 1)) ok = 0;
        for (int j = w.t0; ok && j < w.t1; ++j) {
          const uint32_t gj = g + (uint32_t)(j - w.t0);
          const int sb = (int)(gj & 1), st = (int)((2 * gj) % kParts);
          const uint32_t ph = (2 * gj / kParts) & 1;
          if (!mbar_wait(&c_full[st], ph) || !mbar_wait(&c_full[st + 1], ph) ||
              !mbar_wait(&s_free[sb], ((gj >> 1) & 1) ^ 1)) {
            ok = 0;
            break;
          }
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll
          for (int kc = 0; kc < 4; ++kc)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f8(tmem + kColS + 128u * (uint32_t)sb, desc_add(qd0, kc * kQChunk + ks * 32),
                     desc_add(cd0, kc * kChunk + st * kPart * 128 + ks * 32), idS, (kc | ks) != 0 ? 1u : 0u);
          mma_commit(&s_full[sb]);
          if (j == w.t1 - 1) mma_commit(q_empty);
        }
      }
      ok = __shfl_sync(kFull, ok, 0);
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      ++qw;
      g += (uint32_t)(w.t1 - w.t0);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ O issuer (lane 0)
    constexpr uint32_t idO = idesc_e4m3_f32(64, 256) | (1u << 16);   // B is MN-major
    const uint64_t vd0 = sdesc_mn_sw128(smem_u32(sm + kOffC), kChunk, 1024);
    const uint64_t pd0 = sdesc_k_sw128(smem_u32(sm + kOffP));
    uint32_t g = 0, oi = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const Item w = item_of(it);
      if (w.t0 >= w.t1) continue;
      int ok = 1;
      if (lane == 0) {
        for (int j = w.t0; j < w.t1; ++j) {
          const uint32_t gj = g + (uint32_t)(j - w.t0);
          const int pb = (int)(gj & 1), st = (int)((2 * gj) % kParts);
          if (!mbar_wait(&p_full[pb], (gj >> 1) & 1) ||
              (j == w.t0 && !mbar_wait(o_free, (oi & 1) ^ 1))) {   // the previous item's O has been read
            ok = 0;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
              for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
                  mma_f8(tmem + ((uint32_t)(16 * hh) << 16) + kColO,
                         desc_add(pd0, pb * kPBytes + hl * kPHalf + (2 * p + ks) * 32),
                         desc_add(vd0, 2 * hh * kChunk + ((st + p) * kPart + 32 * ks) * 128), idO,
                         (j > w.t0 || p > 0 || ks > 0 || hl > 0) ? 1u : 0u);
            mma_commit(&t_done[st + p]);
          }
        }
      }
      ok = __shfl_sync(kFull, ok, 0);
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      ++oi;
      g += (uint32_t)(w.t1 - w.t0);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ softmax and epilogue (warps 12-19)
    const int sub = warp & 3, ch = (warp - 12) >> 2;   // lane quarter; half of the tile / of the O columns
    const int half = lane >> 4;                        // which 32 of the warp's 64 entries
    const int hrow = 16 * sub + (lane & 15);           // head of the group
    const uint32_t lane_base = (uint32_t)(32 * sub) << 16;
    float* x_mine = xch + (4 * ch + sub) * 16 + (lane & 15);
    float* x_other = xch + (4 * (ch ^ 1) + sub) * 16 + (lane & 15);
    uint32_t g = 0, qw = 0, xn = 0;   // tiles, items, exchanges
    // value of the partner warp's same head; both warps take part
    auto exchange = [&](float v, float& other) {
      float* slot = x_mine + 128 * (xn & 1);
      if (half == 0) *slot = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_bar[sub]);
      const bool ok = warp_wait(&x_bar[sub], xn & 1);
      other = x_other[128 * (xn & 1)];
      ++xn;
      return ok;
    };
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      const Item w = item_of(it);
      const int head = w.hg * kHeads + hrow;
      if (w.t0 >= w.t1) {   // nothing to see
        if (a.splits > 1) {
          if (ch == 0 && half == 0) a.part_lse[((long long)w.row * a.nh + head) * a.splits + w.split] = -INFINITY;
        } else {
          uint4* o = reinterpret_cast<uint4*>(a.O + (long long)w.row * a.ld_O + (long long)head * kC + 256 * half +
                                              128 * ch);
          for (int i = 0; i < 16; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      bool ok = warp_wait(q_full, qw & 1);
      const float qs = ok ? qs_s[hrow] * a.scale_log2 : 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);
      ++qw;
      // S = ca * own + cb * partner's: the lower lanes own hi and get lo, the upper ones the reverse
      const float ca = half ? qs / kLo : qs, cb = half ? qs : qs / kLo;
      float R = -INFINITY, l = 0.f;    // this lane's running maximum of s, and its sum of 2^(s - R)
      float M = -INFINITY;             // the head's (lagging) maximum of s + e
      const int tiles = w.t1 - w.t0;
      for (int j = 0; ok && j < tiles; ++j) {
        const uint32_t gj = g + (uint32_t)j;
        const int sb = (int)(gj & 1), st = (int)((2 * gj) % kParts) + ch;
        const uint32_t ph = (2 * gj / kParts) & 1;
        if (!warp_wait(&e_full[st], ph) || !warp_wait(&s_full[sb], (gj >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        float s[32];
        const uint32_t col = tmem + lane_base + kColS + 128u * (uint32_t)sb + 64u * (uint32_t)ch;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x0[16], x1[16];
          tmem_ld_x16_pair(col + 16u * b, col + 32u + 16u * b, x0, x1);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float other = __shfl_xor_sync(kFull, half ? x0[k] : x1[k], 16);
            s[16 * b + k] = fmaf(cb, other, ca * (half ? x1[k] : x0[k]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[sb]);
        // entry scales: s to its value, and the maxima of s and of s + e
        uint32_t eb[8];
        {
          const uint4* ep = reinterpret_cast<const uint4*>(e_s + st * kPart + 32 * half);
          const uint4 e0 = ep[0], e1 = ep[1];
          eb[0] = e0.x; eb[1] = e0.y; eb[2] = e0.z; eb[3] = e0.w;
          eb[4] = e1.x; eb[5] = e1.y; eb[6] = e1.z; eb[7] = e1.w;
        }
        const uint32_t vm = valid_s[2 * st + half];
        float smax = -INFINITY, tmax = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t byte = (eb[k >> 2] >> (8 * (k & 3))) & 0xFFu;
          s[k] *= __uint_as_float(byte << 23);   // byte 0 (2^-127) reads as zero
          if (!((vm >> k) & 1u)) s[k] = -INFINITY;
          smax = fmaxf(smax, s[k]);
          tmax = fmaxf(tmax, s[k] + (float)byte);
        }
        tmax = fmaxf(tmax, __shfl_xor_sync(kFull, tmax, 16));
        float other;
        if (!exchange(tmax, other)) { ok = false; break; }
        tmax = fmaxf(tmax, other) - 127.f;
        const bool grow = tmax > M + kGrow;   // also on the first tile with a valid entry
        const float Mn = grow ? tmax : M;
        // P buffer (and, to rescale O, every earlier O product) free?
        if (__any_sync(kFull, grow && j > 0)) {
          const uint32_t gp = 2 * (gj - 1) + 1;
          if (!warp_wait(&t_done[gp % kParts], (gp / kParts) & 1)) { ok = false; break; }
          tc_fence_after();
          const float alpha = grow ? ex2_approx_f32(M - Mn) : 1.f;   // 2^-inf = 0 when nothing was seen
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float v[32];
            const uint32_t ta = tmem + lane_base + kColO + 128u * (uint32_t)ch + 32u * (uint32_t)c;
            tmem_ld_32x32b_x32(ta, v);
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= alpha;
            tmem_st_32x32b_x32(ta, v);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        M = Mn;
        const float Rn = fmaxf(R, smax), Ru = Rn == -INFINITY ? 0.f : Rn;
        l *= ex2_approx_f32(R - Ru);
        R = Rn;
        // w = 2^(s - R) 2^e 2^(R - M + kOff)
        const float f = ex2_approx_f32(fminf(Ru - (M == -INFINITY ? 0.f : M) + kOff, 126.f));
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          hi[q] = 0;
          lo[q] = 0;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int k = 4 * q + 2 * p;
            const float p0 = ex2_approx_f32(s[k] - Ru), p1 = ex2_approx_f32(s[k + 1] - Ru);
            l += p0 + p1;
            const uint32_t b0 = (eb[q] >> (16 * p)) & 0xFFu, b1 = (eb[q] >> (16 * p + 8)) & 0xFFu;
            const __half2 w2 = __floats2half2_rn(p0 * __uint_as_float(b0 << 23) * f, p1 * __uint_as_float(b1 << 23) * f);
            const uint16_t h8 = f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&w2));
            const uint32_t hb = e4m3x2_to_half2(h8);
            const __half2 rest = __hsub2(w2, *reinterpret_cast<const __half2*>(&hb));
            hi[q] |= (uint32_t)h8 << (16 * p);
            lo[q] |= (uint32_t)f16x2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&rest)) << (16 * p);
          }
        }
        const int pb = (int)(gj & 1);
        if (gj >= 2) {   // the P buffer's previous reader
          const uint32_t gp = 2 * (gj - 2) + 1;
          if (!warp_wait(&t_done[gp % kParts], (gp / kParts) & 1)) { ok = false; break; }
        }
        uint8_t* prow = sm + kOffP + pb * kPBytes;
        const int u = 4 * ch + 2 * half;
        *reinterpret_cast<uint4*>(prow + sw128(hrow, u)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(prow + sw128(hrow, u + 1)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4*>(prow + kPHalf + sw128(hrow, u)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(prow + kPHalf + sw128(hrow, u + 1)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[pb]);
      }
      // the head's normaliser relative to M: this lane's, its pair's, the partner warp's
      const bool seen = M != -INFINITY;
      float lm = seen && l > 0.f ? l * ex2_approx_f32(fminf(R - M, 126.f)) : l;
      lm += __shfl_xor_sync(kFull, lm, 16);
      float lo_other = 0.f;
      if (ok && !exchange(lm, lo_other)) ok = false;
      const uint32_t glast = 2 * (g + (uint32_t)tiles - 1) + 1;
      if (!ok || !warp_wait(&t_done[glast % kParts], (glast / kParts) & 1)) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const float lsum = lm + lo_other;
      const float inv = lsum == 0.f ? 0.f : exp2f(-kOff) / lsum;
      // O / l in two passes of 64 columns per lane.  bf16 rows go through 32 staging rows (row = lane: head
      // 16 sub + lane % 16, channels 256 (lane / 16) + 128 ch + 64 p ..) that alias this quarter's rows of P
      // buffer `ch`: its next writers are the two warps of this quarter, after both have met again.
      uint8_t* stage = sm + kOffP + ch * kPBytes + 16 * sub * 128;
      auto stage_row = [&](int r) { return stage + (r >> 4) * kPHalf; };
#pragma unroll 1
      for (int p = 0; p < 2; ++p) {
        float v0[32], v1[32];
        const uint32_t ta = tmem + lane_base + kColO + 128u * (uint32_t)ch + 64u * (uint32_t)p;
        tmem_ld_32x32b_x32_pair(ta, ta + 32u, v0, v1);
        if (p == 1) {   // O is in registers: the next item's O products may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        if (a.splits > 1) {
          float4* o = reinterpret_cast<float4*>(
              a.part_o + (((long long)w.row * a.nh + head) * a.splits + w.split) * kC + 256 * half + 128 * ch + 64 * p);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            o[q] = make_float4(v0[4 * q] * inv, v0[4 * q + 1] * inv, v0[4 * q + 2] * inv, v0[4 * q + 3] * inv);
            o[8 + q] = make_float4(v1[4 * q] * inv, v1[4 * q + 1] * inv, v1[4 * q + 2] * inv, v1[4 * q + 3] * inv);
          }
          continue;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float* vv = u < 4 ? v0 : v1;
          Vec16<__nv_bfloat16> pk;
#pragma unroll
          for (int q = 0; q < 8; ++q) pk.e[q] = __float2bfloat16_rn(vv[8 * (u & 3) + q] * inv);
          *reinterpret_cast<uint4*>(stage_row(lane) + sw128(lane & 15, u)) = pk.u;
        }
        __syncwarp();
        __nv_bfloat16* ob = a.O + (long long)w.row * a.ld_O + (long long)(w.hg * kHeads + 16 * sub) * kC;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), u = lane & 7;
          const uint4 val = *reinterpret_cast<const uint4*>(stage_row(r) + sw128(r & 15, u));
          *reinterpret_cast<uint4*>(ob + (r & 15) * kC + 256 * (r >> 4) + 128 * ch + 64 * p + 8 * u) = val;
        }
        __syncwarp();
      }
      if (a.splits > 1 && ch == 0 && half == 0)
        a.part_lse[((long long)w.row * a.nh + head) * a.splits + w.split] = lsum == 0.f ? -INFINITY : M + log2f(lsum);
      g += (uint32_t)tiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the splits of a (row, head): O = sum_i o_i 2^(lse_i) / sum_i 2^(lse_i),
// the splits added in order.  One CTA of 128 threads per (row, head), four
// channels per thread.
__global__ void __launch_bounds__(128) mqa_f8_join_kernel(const float* part_o, const float* part_lse, int nh, int splits,
                                                          __nv_bfloat16* O, long long ld_O) {
  pdl_prologue_done();
  const long long rh = blockIdx.x;
  const float* lse = part_lse + rh * splits;
  float top = -INFINITY;
  for (int i = 0; i < splits; ++i) top = fmaxf(top, lse[i]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int i = 0; i < splits; ++i) {
    if (lse[i] == -INFINITY) continue;   // nothing seen: part_o was not written
    const float w = exp2f(lse[i] - top);
    const float4 o = reinterpret_cast<const float4*>(part_o + (rh * splits + i) * mqaf8::kC)[threadIdx.x];
    sum += w;
    acc.x = fmaf(w, o.x, acc.x);
    acc.y = fmaf(w, o.y, acc.y);
    acc.z = fmaf(w, o.z, acc.z);
    acc.w = fmaf(w, o.w, acc.w);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long row = rh / nh;
  const int head = (int)(rh - row * nh);
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t*>(&lo);
  u.y = *reinterpret_cast<uint32_t*>(&hi);
  reinterpret_cast<uint2*>(O + row * ld_O + (long long)head * mqaf8::kC)[threadIdx.x] = u;
}

}  // namespace csa
