// Shared-KV MQA over 8-bit entries, eqs. (9)-(11) of "Compressed Sparse
// Attention" (cnblogs), on the 8-bit tensor cores of sm_100a (c = 512, heads
// in groups of 64, bf16 queries).
//
// The entries are E4M3 operands of both products, so the gathered codes feed
// the tensor cores as they are: no widening pass, half the shared memory and
// half the gather of a bf16 tile.  The other operand keeps its precision by
// being split into two 8-bit parts:
//   q = 2^k (hi + lo)   per head, k from the row's maximum: a bf16 value has 8
//                       significant bits, hi (E4M3) takes the upper 4 and lo
//                       (E4M3) the rest, so the split is exact but for values
//                       below 2^-9 of the row's largest (2^-17 of it off);
//   w = hi + lo         the softmax weight times the entry's scale: hi E4M3,
//                       lo E5M2, whose range keeps small weights at 3 bits.
//                       Rounding within 2^-7 (rms 0.12 %, as a bf16 weight).
// A work item is one query row and 64 of its heads (and a range of its parts
// where rows are few).  Per part of 64 selected entries
//   S[128, 64] = [hi; lo] . C^T     M = 128 (64 heads x hi, lo), N = 64
//                                   entries, K = 512: 16 MMAs
//   s = scale_q scale_e (S_hi + S_lo), p = 2^(s - R), u = p scale_e
//   O[64, 512] += w_hi . C + w_lo . C    M = 64, N = 2 x 256 channels, K = 64;
//                                   w = u 2^(R - M + kOff)
// with R a lane's running maximum of s and M the head's (lagging) running
// maximum of s + log2(scale_e), so that the weights use E4M3's range whatever
// the entries' scales are.  The normaliser is summed in fp32 from the
// unrounded probabilities, relative to the maximum of s alone.
//
// The codes sit in shared memory once, [4 chunks of 128 channels][256 ring
// entries][128 bytes] in the 128-byte swizzle: S reads 64 entries as a
// K-major operand, O reads the same bytes MN-major (32 entries = K, 256
// channels = N, two chunks apart by the ring's length).
//
// What bounds it is the chain gather -> S -> softmax -> O -> free of a part
// (the MMAs take 16 x 48 + 8 x 128 = 1.8 K cycles of it, the gather 2.3 K
// beside their shared-memory reads), so the ring holds four parts, each with
// its own S and P buffer, and two groups of four softmax warps take alternate
// parts: while one waits on TMEM, shared memory or the other's M, the other
// computes.  A part takes 2.6 K cycles.  64 decode rows of 128 heads and 2048
// entries run in 62 us (both groups on one 128-entry tile: 67.7; S over
// pairs of parts: 68.3; eight warps that gather and split q: 71.2), 8192
// packed rows of 64 heads and up to 512 entries in 717 to 772 us (717 where the
// bf16 kernel took 824 over the same entries read back).
//
// TMEM (512 columns): O in columns 0-255 (channels 0-255 in the lower 16
// lanes of every lane quarter, 256-511 in the upper 16); four S buffers of 64
// columns.  Lane quarter `sub` holds heads 16 sub .. + 15: their hi rows in
// its lower 16 lanes, their lo rows in the upper 16.
//
// Warps (20): 0-3 gather codes (16-byte cp.async, one entry per warp and
// instruction) and split half of q; 4-7 split the other half; 8 fetches the
// entries' scales; 9 issues S, 10 issues O (one thread each); 11 owns TMEM and posts
// the work items ahead of their consumers; 12-19 softmax and epilogue.
// Every wait is bounded (sm100::mbar_wait); the groups meet on mbarriers,
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
  int parts_per_split;
  float* part_o;                            // splits > 1: [rows, nh, splits, 512]
  float* part_lse;                          //             [rows, nh, splits], base 2; -inf: nothing seen
};

namespace mqaf8 {
constexpr int kC = 512, kHeads = 64, kPart = 64, kParts = 4;
constexpr int kChunk = kParts * kPart * 128;      // ring bytes of one 128-channel chunk
constexpr int kQChunk = 128 * 128;                // q: 128 rows x 128 channels
constexpr int kPBytes = 64 * 128;                 // P of a part: 64 heads x (64 hi | 64 lo)
constexpr int kOffC = 4 * kQChunk;
constexpr int kOffP = kOffC + 4 * kChunk;         // kParts P buffers; the epilogue's staging rows between items
constexpr int kOffE = kOffP + kParts * kPBytes;   // scale (fp32) of each ring entry
constexpr int kOffX = kOffE + kParts * kPart * 4; // xch: [2 groups][64 heads] pairs of fp32
constexpr int kOffS = kOffX + 2 * kHeads * 8;     // q scale of each head
constexpr int kOffMisc = kOffS + kHeads * 4;
constexpr size_t kSmem = kOffMisc + 768;          // the swizzled tiles need a base aligned to 1024 bytes
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr int kItems = 4;                         // item descriptors in flight
constexpr int kReaders = 4 + 4 + 3 + 8;           // warps that read each of them
constexpr int kThreads = 640;
constexpr int kMaxSplits = 64;                    // of a (row, head group)
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;
// w <= 2^(kOff + kGrow) = 362 < 448: the running maximum may lag by kGrow, and
// the largest weight stays above 2^kOff.  A rescale of O costs a part's time
// (it waits for the products in flight), so kGrow is most of E4M3's range.
constexpr float kOff = 3.5f, kGrow = 5.f;
// M counts no scale below this, so that M >= R - 123 for every maximum R of the
// scores and 2^(R - M + kOff) <= 2^126.5 is in fp32's range.  Where all of a
// head's scales are smaller its largest weight is 2^(-127 + 118 + kOff) = 2^-5.5
// or more, which hi still holds as a normal number.
constexpr float kMinScale = 0x1p-118f;
}  // namespace mqaf8

// Parts of 64 slots up to the row's last valid slot (0 <= s < avail), by a
// whole warp.  The row is read from its end, 512 slots at a time, so a full row costs one memory latency.
__device__ __forceinline__ int mqa_f8_nparts(const int* ir, int topk, int avail) {
  const int lane = threadIdx.x & 31;
  for (int j0 = ((topk - 1) / 512) * 512; j0 >= 0; j0 -= 512) {
    int v[16], last = -1;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const int j = j0 + 32 * u + lane;
      v[u] = j < topk ? __ldg(ir + j) : -1;
    }
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      if (v[u] >= 0 && v[u] < avail) last = j0 + 32 * u + lane;
      else if (v[u] != -1) flag_status(kStatusBadIndex);   // (those before the last valid slot: the scale warp too)
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last >= 0) return last / mqaf8::kPart + 1;
  }
  return 0;
}

// Four fp16 values (two pairs) as hi + lo, one byte each: hi their E4M3
// rounding, lo the rest in E4M3 (or E5M2).  The rest is exact in fp16, so lo
// also holds what hi lost to E4M3's range.
#define CSA_SPLIT4(LO_TYPE)                                       \
  asm("{\n\t.reg .b16 a, b;\n\t.reg .b32 p, q;\n\t"             \
      "cvt.rn.satfinite.e4m3x2.f16x2 a, %2;\n\t"                  \
      "cvt.rn.satfinite.e4m3x2.f16x2 b, %3;\n\t"                  \
      "mov.b32 %0, {a, b};\n\t"                                   \
      "cvt.rn.f16x2.e4m3x2 p, a;\n\t"                             \
      "cvt.rn.f16x2.e4m3x2 q, b;\n\t"                             \
      "sub.f16x2 p, %2, p;\n\t"                                   \
      "sub.f16x2 q, %3, q;\n\t"                                   \
      "cvt.rn.satfinite." LO_TYPE ".f16x2 a, p;\n\t"              \
      "cvt.rn.satfinite." LO_TYPE ".f16x2 b, q;\n\t"              \
      "mov.b32 %1, {a, b};\n\t}"                                  \
      : "=r"(hi), "=r"(lo)                                        \
      : "r"(h0), "r"(h1))
__device__ __forceinline__ void split4_e4m3(uint32_t h0, uint32_t h1, uint32_t& hi, uint32_t& lo) {
  CSA_SPLIT4("e4m3x2");
}
__device__ __forceinline__ void split4_e4m3_e5m2(uint32_t h0, uint32_t h1, uint32_t& hi, uint32_t& lo) {
  CSA_SPLIT4("e5m2x2");
}
#undef CSA_SPLIT4
// Two fp32 values rounded to an fp16 pair.
__device__ __forceinline__ uint32_t to_half2(float2 x) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 consecutive fp32 TMEM columns of this thread's lane from `t0` and 16 from
// `t1`, with a single wait.
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

using f8::add2;
using f8::mul2;
using f8::pk2;
using f8::upk2;
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x like ex2_approx_f32, with subnormal results.
__device__ __forceinline__ float ex2_approx_all_f32(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx_f32(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A work item: its row, head group and split, and the parts [p0, p1) of the
// row that it covers (none where p0 >= p1).
struct MqaF8Item {
  int row, hg, split, p0, p1, avail;
  long long base;
};

// Splits the query rows of heads `h0` .. h0 + heads - 1 of an item's 64 into
// the swizzled q tile, by a whole warp (a lane 16 channels of each head): two
// heads at a time, so that one's reduction and conversions fill the other's
// latencies, with the next two on their way.  heads is a multiple of 4.
// `empty`: the tile's release, waited for before the first store.  Out of line:
// both the q warps and, for a CTA's first item, the softmax warps run it.
__device__ __noinline__ bool mqa_f8_split_q(const __nv_bfloat16* q64, int h0, int heads, uint8_t* sm, float* qs_s,
                                            uint64_t* empty, uint32_t parity) {
  using namespace mqaf8;
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* qrow = q64 + (long long)h0 * kC + 16 * lane;
  uint4 raw[2][2][2];   // [pair of heads in flight][head][16 bytes]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) raw[i >> 1][i & 1][u] = __ldg(reinterpret_cast<const uint4*>(qrow + i * kC) + u);
  uint8_t* dst = sm + (lane >> 3) * kQChunk;
#pragma unroll 1
  for (int i0 = 0; i0 < heads; i0 += 4) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int i = i0 + 2 * b;
      uint32_t rw[2][8], ex[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 r0 = raw[b][k][0], r1 = raw[b][k][1];
        rw[k][0] = r0.x; rw[k][1] = r0.y; rw[k][2] = r0.z; rw[k][3] = r0.w;
        rw[k][4] = r1.x; rw[k][5] = r1.y; rw[k][6] = r1.z; rw[k][7] = r1.w;
        if (i + 4 < heads)
#pragma unroll
          for (int u = 0; u < 2; ++u) raw[b][k][u] = __ldg(reinterpret_cast<const uint4*>(qrow + (i + 4 + k) * kC) + u);
        __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);   // the larger magnitude of each half
#pragma unroll
        for (int e = 0; e < 8; ++e) m2 = __hmax2(m2, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&rw[k][e])));
        const uint32_t m = *reinterpret_cast<const uint32_t*>(&m2);
        ex[k] = max(m & 0xFFFFu, m >> 16);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) ex[k] = max(__reduce_max_sync(0xffffffffu, ex[k]) >> 7, 8u);
      uint32_t hi[2][4], lo[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // 2^-k with the largest value in [128, 256).  An infinite or NaN
        // value gives a NaN lo, and with it NaN scores.
        const float inv = __uint_as_float((261u - ex[k]) << 23);
        const uint64_t inv2 = pk2(inv, inv);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t h[2];   // exact in fp16: 8 bits, below 256
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t wd = rw[k][2 * q + p];
            h[p] = to_half2(upk2(mul2(pk2(__uint_as_float(wd << 16), __uint_as_float(wd & 0xFFFF0000u)), inv2)));
          }
          split4_e4m3(h[0], h[1], hi[k][q], lo[k][q]);
        }
      }
      if (i == 0 && !sm100::warp_wait_small(empty, parity)) return false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int head = h0 + i + k, r = 32 * (head >> 4) + (head & 15);
        *reinterpret_cast<uint4*>(dst + sw128(r, lane & 7)) = make_uint4(hi[k][0], hi[k][1], hi[k][2], hi[k][3]);
        *reinterpret_cast<uint4*>(dst + sw128(r + 16, lane & 7)) = make_uint4(lo[k][0], lo[k][1], lo[k][2], lo[k][3]);
        if (lane == 0) qs_s[head] = __uint_as_float((ex[k] - 7u) << 23);
      }
    }
  }
  sm100::fence_proxy_async_smem();
  __syncwarp();
  return true;
}

__global__ void __launch_bounds__(mqaf8::kThreads, 1) mqa_f8_tc_kernel(MqaF8TcArgs a) {
  using namespace sm100;
  using namespace mqaf8;
  constexpr uint32_t kFull = 0xffffffffu;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {   // the declared alignment; the tiles' swizzle relies on it
    flag_status(kStatusBounds);
    return;
  }
  float* e_s = reinterpret_cast<float*>(sm + kOffE);
  float2* xch = reinterpret_cast<float2*>(sm + kOffX);
  float* qs_s = reinterpret_cast<float*>(sm + kOffS);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + kOffMisc);
  uint64_t* q_empty = q_full + 1;         // the item's last S done, and every softmax warp has its q scales
  uint64_t* c_full = q_empty + 1;         // [kParts] codes landed
  uint64_t* e_full = c_full + kParts;     // [kParts] scales and validity written
  uint64_t* t_done = e_full + kParts;     // [kParts] O product of the part done: frees its ring entries and P buffer
  uint64_t* s_full = t_done + kParts;     // [kParts]
  uint64_t* s_free = s_full + kParts;     // [kParts]
  uint64_t* p_full = s_free + kParts;     // [kParts]
  uint64_t* o_free = p_full + kParts;
  uint64_t* x_bar = o_free + 1;           // [2 groups][4 lane quarters] a value posted in xch
  uint64_t* it_full = x_bar + 8;          // [kItems] item descriptor posted
  uint64_t* it_free = it_full + kItems;   // [kItems] read by its kReaders consumer warps
  MqaF8Item* item_s = reinterpret_cast<MqaF8Item*>(it_free + kItems);
  uint32_t* valid_s = reinterpret_cast<uint32_t*>(item_s + kItems);   // [kParts][2] validity of the ring entries
  uint32_t* tmem_slot = valid_s + 2 * kParts;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hgroups = a.nh / kHeads;
  const int per_row = hgroups * a.splits;
  const int items = a.rows * per_row;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 16);
    mbar_init(q_empty, 1 + 8);
    for (int s = 0; s < kParts; ++s) {
      mbar_init(&c_full[s], 128);
      mbar_init(&e_full[s], 1);
      mbar_init(&t_done[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
      mbar_init(&p_full[s], 4);
    }
    mbar_init(o_free, 8);
    for (int s = 0; s < 8; ++s) mbar_init(&x_bar[s], 1);
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&it_full[s], 1);
      mbar_init(&it_free[s], kReaders);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 11) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_prologue_done();
  const uint32_t tmem = *tmem_slot;

  // The n-th item of this CTA, as warp 11 posted it (a whole warp; false: a wait ran out).
  auto item_of = [&](uint32_t n, MqaF8Item& w) {
    const int slot = (int)(n % kItems);
    const bool ok = warp_wait_small(&it_full[slot], (n / kItems) & 1);
    w = item_s[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_free[slot]);
    if (!ok && lane == 0) *abort_flag = 1;
    return ok;
  };

  if (warp < 4) {
    // ------------------------------------------------------------ gather (warps 0-3)
    // entry warp + 4 i of a part per instruction, a lane 16 bytes; slots fetched one part ahead
    uint32_t g = 0, qw = 0, n = 0;   // ring parts, items with parts, items
    bool ok = true;
    const uint32_t ring = smem_u32(sm + kOffC + (lane >> 3) * kChunk);
    const uint32_t swz0 = sw128(warp, lane & 7), swz1 = sw128(warp + 4, lane & 7);
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      if (w.p0 >= w.p1) continue;
      const int* ir = a.idx + (long long)w.row * a.topk;
      if (qw++ > 0) {   // their share of q (see the q warps)
        const __nv_bfloat16* q64 = a.q + (long long)w.row * a.ld_q + (long long)(w.hg * kHeads) * kC;
        if (!mqa_f8_split_q(q64, 32 + 8 * warp, 8, sm, qs_s, q_empty, qw & 1)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive(q_full);
          mbar_arrive(q_full);
        }
      }
      const long long n_ent = rowmap_entries(a.rm, a.rows);
      auto slot = [&](int p) {
        const int e = p * kPart + warp + 4 * lane;
        return lane < 16 && e < a.topk ? __ldg(ir + e) : -1;
      };
      const uint8_t* src0 = a.codes + w.base * kC + 16 * lane;
      int next = slot(w.p0);
      for (int p = w.p0; p < w.p1; ++p, ++g) {
        const int st = (int)(g % kParts);
        const int mine = next;
        next = p + 1 < w.p1 ? slot(p + 1) : -1;
        if (!warp_wait_small(&t_done[st], ((g / kParts) & 1) ^ 1)) { ok = false; break; }
        // rows warp + 4 i: two swizzle phases, 1024 bytes every other row
        const uint32_t dst = ring + (uint32_t)(st * kPart * 128);
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int s = __shfl_sync(kFull, mine, i);
          const bool v = (unsigned)s < (unsigned)w.avail && dcheck(w.base + s < n_ent);
          cp_async16_to(dst + ((i & 1) ? swz1 : swz0) + (uint32_t)(i >> 1) * 1024u, v ? src0 + (long long)s * kC : a.codes,
                        v ? 16u : 0u);
        }
        cp_async_arrive_noinc(&c_full[st]);
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    cp_async_wait_all();
  } else if (warp < 8) {
    // ------------------------------------------------------------ q split (warps 4-7)
    // 8 heads each, the gather warps taking the other 32 (the next item's S
    // waits for q, so its first entries can wait too); of the first item 4
    // each, the softmax warps taking 48 (they have nothing else to do yet)
    uint32_t qw = 0, n = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      if (w.p0 >= w.p1) continue;
      const __nv_bfloat16* q64 = a.q + (long long)w.row * a.ld_q + (long long)(w.hg * kHeads) * kC;
      const bool first = qw == 0;
      const int heads = first ? 4 : 8;
      if (!mqa_f8_split_q(q64, (warp - 4) * heads, heads, sm, qs_s, q_empty, (qw & 1) ^ 1)) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      if (lane == 0)
        for (int u = 0; u < (first ? 1 : 2); ++u) mbar_arrive(q_full);
      ++qw;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ scales and validity
    uint32_t g = 0, n = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      const int* ir = a.idx + (long long)w.row * a.topk;
      bool ok = true;
      for (int p = w.p0; p < w.p1; ++p, ++g) {
        const int st = (int)(g % kParts);
        bool v[2];
        uint32_t b[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int e = p * kPart + 32 * u + lane;
          const int s = e < a.topk ? __ldg(ir + e) : -1;
          v[u] = s >= 0 && s < w.avail;
          if (!v[u] && s != -1) flag_status(kStatusBadIndex);
          b[u] = v[u] ? __ldg(a.scales + w.base + s) : 0u;
        }
        if (!warp_wait_small(&t_done[st], ((g / kParts) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          e_s[st * kPart + 32 * u + lane] = f8::scale_value(b[u]);
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
    // ------------------------------------------------------------ S issuer
    constexpr uint32_t idS = idesc_e4m3_f32(128, kPart);
    const uint32_t qd0 = sdesc_lo(smem_u32(sm), 16), cd0 = sdesc_lo(smem_u32(sm + kOffC), 16);
    uint32_t g = 0, qw = 0, n = 0;   // parts, items with parts, items
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      const int np = w.p1 - w.p0;
      if (np <= 0) continue;
      bool ok = warp_wait_small(q_full, qw & 1);
      for (int j = 0; ok && j < np; ++j, ++g) {
        const int st = (int)(g % kParts);
        const uint32_t ph = (g / kParts) & 1;
        if (!warp_wait_small(&c_full[st], ph) || !warp_wait_small(&s_free[st], ph ^ 1)) { ok = false; break; }
        fence_proxy_async_smem();
        tc_fence_after();
        if (lane == 0) {
          const uint32_t cd = cd0 + (uint32_t)(st * kPart * 128 >> 4);
#pragma unroll
          for (int kc = 0; kc < 4; ++kc)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f8(tmem + kColS + (uint32_t)(kPart * st), qd0 + (uint32_t)((kc * kQChunk + ks * 32) >> 4),
                     cd + (uint32_t)((kc * kChunk + ks * 32) >> 4), sdesc_hi(1024), sdesc_hi(1024), idS,
                     (kc | ks) != 0 ? 1u : 0u);
          mma_commit(&s_full[st]);
          if (j == np - 1) mma_commit(q_empty);
        }
        __syncwarp();
      }
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      ++qw;
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ O issuer
    constexpr uint32_t idHi = idesc_e4m3_f32(64, 256) | (1u << 16);   // B is MN-major
    constexpr uint32_t idLo = idHi | (1u << 7);                       // A is E5M2
    const uint32_t vd0 = sdesc_lo(smem_u32(sm + kOffC), kChunk), pd0 = sdesc_lo(smem_u32(sm + kOffP), 16);
    uint32_t g = 0, oi = 0, n = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      const int np = w.p1 - w.p0;
      if (np <= 0) continue;
      bool ok = warp_wait_small(o_free, (oi & 1) ^ 1);   // the previous item's O has been read
      for (int j = 0; ok && j < np; ++j, ++g) {
        const int st = (int)(g % kParts);
        if (!warp_wait_small(&p_full[st], (g / kParts) & 1)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          const uint32_t pd = pd0 + (uint32_t)(st * kPBytes >> 4), vd = vd0 + (uint32_t)(st * kPart * 128 >> 4);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int hl = 0; hl < 2; ++hl)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
                mma_f8(tmem + ((uint32_t)(16 * hh) << 16) + kColO, pd + (uint32_t)((64 * hl + 32 * ks) >> 4),
                       vd + (uint32_t)((2 * hh * kChunk + 32 * ks * 128) >> 4), sdesc_hi(1024), sdesc_hi(1024),
                       hl ? idLo : idHi, (j > 0 || ks > 0 || hl > 0) ? 1u : 0u);
          mma_commit(&t_done[st]);
        }
        __syncwarp();
      }
      if (!ok) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      ++oi;
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------ item scheduler
    // Rows run last first: they see the most entries.  A lane looks up the
    // row of one of 32 items; each item's index row is then scanned for its
    // parts, up to kItems items ahead of their consumers.
    uint32_t n = 0;
    bool ok = true;
    for (unsigned it0 = blockIdx.x; it0 < (unsigned)items && ok; it0 += 32u * gridDim.x) {
      const unsigned mine = it0 + (unsigned)lane * gridDim.x;   // items + 32 CTAs per SM stay below 2^32
      int row = 0, avail = 0, hg = 0, split = 0;
      long long base = 0;
      if (mine < (unsigned)items) {
        const unsigned q = mine / (unsigned)per_row, r = mine - q * (unsigned)per_row;
        row = a.rows - 1 - (int)q;
        hg = (int)(r / (unsigned)a.splits);
        split = (int)(r - (unsigned)hg * (unsigned)a.splits);
        row_entries(a.rm, row, base, avail);
      }
#pragma unroll 1
      for (unsigned u = 0; u < 32 && it0 + u * gridDim.x < (unsigned)items; ++u, ++n) {
        if (warp_aborted(abort_flag)) { ok = false; break; }
        MqaF8Item w;
        w.row = __shfl_sync(kFull, row, u);
        w.avail = __shfl_sync(kFull, avail, u);
        w.base = __shfl_sync(kFull, base, u);
        w.hg = __shfl_sync(kFull, hg, u);
        w.split = __shfl_sync(kFull, split, u);
        const int parts = mqa_f8_nparts(a.idx + (long long)w.row * a.topk, a.topk, w.avail);
        w.p0 = w.split * a.parts_per_split;
        w.p1 = min(parts, w.p0 + a.parts_per_split);
        if (w.p0 < w.p1) {   // 64 heads x 1 KB of q on their way to L2 (from memory at prefill)
          const __nv_bfloat16* q = a.q + (long long)w.row * a.ld_q + (long long)(w.hg * kHeads) * kC + 64 * lane;
#pragma unroll 4
          for (int i = 0; i < 16; ++i) prefetch_l2(q + i * 4 * kC);
        }
        const int slot = (int)(n % kItems);
        if (!warp_wait_small(&it_free[slot], ((n / kItems) & 1) ^ 1)) {
          if (lane == 0) *abort_flag = 1;
          ok = false;
          break;
        }
        if (lane == 0) {
          item_s[slot] = w;
          mbar_arrive(&it_full[slot]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and epilogue (warps 12-19)
    const int sub = warp & 3, grp = (warp - 12) >> 2;   // lane quarter; parts of this parity / half of the O columns
    const int half = lane >> 4;                         // which 32 of a part's entries
    const int hrow = 16 * sub + (lane & 15);            // head of the group
    const uint32_t lane_base = (uint32_t)(32 * sub) << 16;
    uint32_t g = 0, qw = 0, n = 0;      // parts, items with parts, items
    uint32_t seen_n = 0;                // values of the other group's warp read so far
    // Values go from a group's warp to the other group's warp of the same
    // lane quarter and come back in turn, so one slot each is enough.
    auto post = [&](float v, float u) {
      if (half == 0) xch[grp * kHeads + hrow] = make_float2(v, u);
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_bar[4 * grp + sub]);
    };
    auto receive = [&](float2& v) {
      const bool ok = warp_wait_small(&x_bar[4 * (grp ^ 1) + sub], seen_n & 1);
      ++seen_n;
      v = xch[(grp ^ 1) * kHeads + hrow];
      return ok;
    };
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
      if (warp_aborted(abort_flag)) break;
      MqaF8Item w;
      if (!item_of(n++, w)) break;
      const int head = w.hg * kHeads + hrow;
      if (w.p0 >= w.p1) {   // nothing to see
        if (a.splits > 1) {
          if (grp == 0 && half == 0) a.part_lse[((long long)w.row * a.nh + head) * a.splits + w.split] = -INFINITY;
        } else {
          uint4* o = reinterpret_cast<uint4*>(a.O + (long long)w.row * a.ld_O + (long long)head * kC + 256 * half +
                                              128 * grp);
          for (int i = 0; i < 16; ++i) o[i] = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      bool ok = true;
      if (qw == 0) {   // a share of the first item's q
        const __nv_bfloat16* q64 = a.q + (long long)w.row * a.ld_q + (long long)(w.hg * kHeads) * kC;
        if (warp < 16) ok = mqa_f8_split_q(q64, 16 + 8 * (warp - 12), 8, sm, qs_s, q_empty, 1u);
        else ok = mqa_f8_split_q(q64, 48 + 4 * (warp - 16), 4, sm, qs_s, q_empty, 1u);
        if (lane == 0) {
          mbar_arrive(q_full);
          if (warp < 16) mbar_arrive(q_full);
        }
      }
      ok = ok && warp_wait_small(q_full, qw & 1);
      const float qs = ok ? qs_s[hrow] * a.scale_log2 : 0.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty);
      ++qw;
      const uint64_t qs2 = pk2(qs, qs);
      float R = -INFINITY, l = 0.f;    // this lane's running maximum of s, and its sum of 2^(s - R)
      float M = -INFINITY;             // the head's (lagging) maximum of s + log2(scale)
      float2 seen;                     // what the other group posted
      const int np = w.p1 - w.p0;
      const uint32_t glast = g + (uint32_t)np - 1;
      for (int j = (int)((g ^ (uint32_t)grp) & 1); ok && j < np; j += 2) {
        const uint32_t gj = g + (uint32_t)j;
        const int st = (int)(gj % kParts);
        const uint32_t ph = (gj / kParts) & 1;
        if (!warp_wait_small(&e_full[st], ph) || !warp_wait_small(&s_full[st], ph)) { ok = false; break; }
        tc_fence_after();
        uint64_t v[16];   // s of this lane's 32 entries, in pairs
        const uint32_t col = tmem + lane_base + kColS + (uint32_t)(kPart * st);
        const ulonglong2* ep = reinterpret_cast<const ulonglong2*>(e_s + st * kPart + 32 * half);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x0[16], x1[16];
          tmem_ld_x16_pair(col + 16u * b, col + 32u + 16u * b, x0, x1);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float o0 = __shfl_xor_sync(kFull, half ? x0[k] : x1[k], 16);
            const float o1 = __shfl_xor_sync(kFull, half ? x0[k + 1] : x1[k + 1], 16);
            v[8 * b + k / 2] =   // hi + lo: one's own column plus the partner lane's
                mul2(qs2, add2(pk2(o0, o1), half ? pk2(x1[k], x1[k + 1]) : pk2(x0[k], x0[k + 1])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[st]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const ulonglong2 e = ep[k];
          v[2 * k] = mul2(v[2 * k], e.x);
          v[2 * k + 1] = mul2(v[2 * k + 1], e.y);
        }
        const uint32_t vm = valid_s[2 * st + half];
        if (vm != kFull) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 x = upk2(v[k]);
            if (!((vm >> (2 * k)) & 1u)) x.x = -INFINITY;
            if (!((vm >> (2 * k + 1)) & 1u)) x.y = -INFINITY;
            v[k] = pk2(x.x, x.y);
          }
        }
        // probabilities relative to this lane's running maximum R, their sum, and
        // u = p scale, whose maximum gives that of s + log2(scale)
        float Rn = R;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 x = upk2(v[k]);
          Rn = max3(Rn, x.x, x.y);
        }
        const float Ru = Rn == -INFINITY ? 0.f : Rn;
        l *= ex2_approx_f32(R - Ru);
        R = Rn;
        float umax = 0.f;
        {
          const uint64_t mr2 = pk2(-Ru, -Ru);
          uint64_t l2 = pk2(l, 0.f);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const ulonglong2 e = ep[k / 2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float2 x = upk2(add2(v[k + q], mr2));
              const uint64_t p = pk2(ex2_approx_f32(x.x), ex2_approx_f32(x.y));
              l2 = add2(l2, p);
              v[k + q] = mul2(p, q ? e.y : e.x);
              const float2 u = upk2(v[k + q]);
              umax = max3(umax, u.x, u.y);
            }
          }
          const float2 ls = upk2(l2);
          l = ls.x + ls.y;
        }
        float tmax = Rn + lg2_approx_f32(fmaxf(umax, kMinScale));   // -inf while this lane has seen nothing
        tmax = fmaxf(tmax, __shfl_xor_sync(kFull, tmax, 16));
        if (j > 0) {   // M after the part before
          if (!receive(seen)) { ok = false; break; }
          M = seen.x;
        }
        const bool grow = tmax > M + kGrow;   // also on the first part with a valid entry
        const float Mn = grow ? tmax : M;
        post(Mn, 0.f);
        if (__any_sync(kFull, grow && j > 0)) {   // rescale O: its earlier products must have completed
          const uint32_t gp = gj - 1;
          if (!warp_wait_small(&t_done[gp % kParts], (gp / kParts) & 1)) { ok = false; break; }
          tc_fence_after();
          const float alpha = grow ? ex2_approx_f32(M - Mn) : 1.f;   // 2^-inf = 0 when nothing was seen
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float o[32];
            const uint32_t ta = tmem + lane_base + kColO + 32u * (uint32_t)c;
            tmem_ld_32x32b_x32(ta, o);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] *= alpha;
            tmem_st_32x32b_x32(ta, o);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        M = Mn;
        // w = u 2^(R - M + kOff), as hi + lo.  The part's P buffer is free: its S could only be issued on ring
        // entries that the O product of four parts before, the buffer's last reader, had released.
        // (f is as small as 2^-123 times the lane's part of the softmax where scales are large: subnormal, with u above
        // one.  The bound on f is for lanes that have seen nothing, whose u is 0.)
        const float f = ex2_approx_all_f32(fminf(Ru - (M == -INFINITY ? 0.f : M) + kOff, 127.f));
        const uint64_t f2 = pk2(f, f);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          split4_e4m3_e5m2(to_half2(upk2(mul2(v[2 * q], f2))), to_half2(upk2(mul2(v[2 * q + 1], f2))), hi[q], lo[q]);
        uint8_t* prow = sm + kOffP + st * kPBytes;
        *reinterpret_cast<uint4*>(prow + sw128(hrow, 2 * half)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(prow + sw128(hrow, 2 * half + 1)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        *reinterpret_cast<uint4*>(prow + sw128(hrow, 4 + 2 * half)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4*>(prow + sw128(hrow, 5 + 2 * half)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[st]);
      }
      // The head's M is that of the item's last part.  Its normaliser is that of all its lanes' (R, l), relative to
      // the largest R: M says nothing of it, as an entry's score and its scale are independent (a zero entry has the
      // score 0 and the scale 2^-127).
      const bool last_mine = (int)(glast & 1) == grp;
      if (ok && !last_mine) {
        ok = receive(seen);
        M = seen.x;
      }
      const float Rh = fmaxf(R, __shfl_xor_sync(kFull, R, 16));
      float lh = l * ex2_approx_f32(R - (Rh == -INFINITY ? 0.f : Rh));
      lh += __shfl_xor_sync(kFull, lh, 16);
      seen = make_float2(-INFINITY, 0.f);
      if (ok && !last_mine) post(Rh, lh);
      if (ok) ok = receive(seen);
      if (ok && last_mine) post(Rh, lh);
      if (!ok || !warp_wait_small(&t_done[glast % kParts], (glast / kParts) & 1)) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const float top = fmaxf(Rh, seen.x), ref = top == -INFINITY ? 0.f : top;
      const float lmine = lh * ex2_approx_f32(Rh - ref), lother = seen.y * ex2_approx_f32(seen.x - ref);
      const float lsum = grp == 0 ? lmine + lother : lother + lmine;   // the same sum in both groups
      const float inv = lsum == 0.f ? 0.f : exp2f(M - ref - kOff) / lsum;   // O holds sums of 2^(s - M + kOff) scale code
      // O / l in four passes of 32 columns per lane, through 32 staging rows (row = lane: head 16 sub + lane % 16,
      // channels 256 (lane / 16) + 128 grp + 32 p ..) that alias this quarter's rows of the P buffers grp and
      // grp + 2, which only this warp writes: 64 bytes a row in bf16, 128 bytes in fp32 (a split's partial output).
      uint8_t* stage = sm + kOffP + grp * kPBytes + 16 * sub * 128;
      __nv_bfloat16* ob = a.O + (long long)w.row * a.ld_O + (long long)(w.hg * kHeads + 16 * sub) * kC + 128 * grp;
      float* po = a.part_o + (((long long)w.row * a.nh + w.hg * kHeads + 16 * sub) * a.splits + w.split) * kC + 128 * grp;
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        float v[32];
        tmem_ld_32x32b_x32(tmem + lane_base + kColO + 128u * (uint32_t)grp + 32u * (uint32_t)p, v);
        if (p == 3) {   // O is in registers: the next item's O products may start
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        if (a.splits > 1) {
          auto row = [&](int r) { return stage + (r >> 4) * (2 * kPBytes); };
#pragma unroll
          for (int u = 0; u < 8; ++u)
            *reinterpret_cast<float4*>(row(lane) + sw128(lane & 15, u)) =
                make_float4(v[4 * u] * inv, v[4 * u + 1] * inv, v[4 * u + 2] * inv, v[4 * u + 3] * inv);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), u = lane & 7;
            const float4 val = *reinterpret_cast<const float4*>(row(r) + sw128(r & 15, u));
            *reinterpret_cast<float4*>(po + (long long)(r & 15) * a.splits * kC + 256 * (r >> 4) + 32 * p + 4 * u) = val;
          }
          __syncwarp();
          continue;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          Vec16<__nv_bfloat16> pk;
#pragma unroll
          for (int q = 0; q < 8; ++q) pk.e[q] = __float2bfloat16_rn(v[8 * u + q] * inv);
          *reinterpret_cast<uint4*>(stage + sw64(lane, u)) = pk.u;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2), u = lane & 3;
          const uint4 val = *reinterpret_cast<const uint4*>(stage + sw64(r, u));
          *reinterpret_cast<uint4*>(ob + (r & 15) * kC + 256 * (r >> 4) + 32 * p + 8 * u) = val;
        }
        __syncwarp();
      }
      if (a.splits > 1 && grp == 0 && half == 0)
        a.part_lse[((long long)w.row * a.nh + head) * a.splits + w.split] =
            lsum == 0.f ? -INFINITY : ref + log2f(lsum);   // 0: no valid entry
      g += (uint32_t)np;
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
// channels per thread.  The work is all memory latency (32 splits of 2 KB), so
// the weights are read by lanes of a warp at once and eight splits' values are
// in flight.
__global__ void __launch_bounds__(128) mqa_f8_join_kernel(const float* part_o, const float* part_lse, int nh, int splits,
                                                          __nv_bfloat16* O, long long ld_O) {
  __shared__ float w_s[mqaf8::kMaxSplits];
  pdl_prologue_done();
  const long long rh = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const float4* o = reinterpret_cast<const float4*>(part_o + rh * splits * mqaf8::kC) + threadIdx.x;
  float lse[mqaf8::kMaxSplits / 32], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < mqaf8::kMaxSplits / 32; ++i) {
    lse[i] = 32 * i + lane < splits ? part_lse[rh * splits + 32 * i + lane] : -INFINITY;
    top = fmaxf(top, lse[i]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (threadIdx.x < 32) {
#pragma unroll
    for (int i = 0; i < mqaf8::kMaxSplits / 32; ++i)   // 0 where nothing was seen (and part_o was not written)
      w_s[32 * i + lane] = lse[i] == -INFINITY ? 0.f : exp2f(lse[i] - top);
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int i0 = 0; i0 < splits; i0 += 8) {
    float4 v[8];
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = i0 + i < splits ? w_s[i0 + i] : 0.f;
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (w[i] != 0.f) v[i] = o[(long long)(i0 + i) * (mqaf8::kC / 4)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += w[i];
      acc.x = fmaf(w[i], v[i].x, acc.x);
      acc.y = fmaf(w[i], v[i].y, acc.y);
      acc.z = fmaf(w[i], v[i].z, acc.z);
      acc.w = fmaf(w[i], v[i].w, acc.w);
    }
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
