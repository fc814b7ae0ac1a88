// The load producer of the 8-bit product: which stage of the ring each K block
// of its work units goes to, and which loads are waited for when a wait runs
// out.  Plain C++ over the operations that it is given, so that the host can
// run it against a model of the barriers.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define CSA_RING_FN __device__ __forceinline__
#else
#define CSA_RING_FN inline
#endif

namespace csa {

// Round (from 0) of the last of `filled` fills that went to `stage`; -1: none did.
CSA_RING_FN int ring_last_round(uint32_t filled, int stage, int stages) {
  return (uint32_t)stage < filled ? (int)((filled - 1u - (uint32_t)stage) / (uint32_t)stages) : -1;
}

// Fills the ring of kGroups groups of four stages, in order, for the work
// units first, first + step .. below total; unit u is K blocks
// [u % k_split * kbs, + kbs) of tile u / k_split.  Groups are whole: blocks
// past a unit's end are filled empty.  Ops:
//   aborted()                  a wait of some role ran out
//   abort()                    one of this role did
//   tile(t)                    the blocks that follow are tile t's
//   wait_empty(stage, parity)  false: the wait ran out
//   fill(stage, kb, real)      starts the loads of K block kb, or (not real) completes the stage without any
//   wait_full(stage, parity)   waits for the loads of a fill
template <int kGroups, typename Ops>
CSA_RING_FN void f8_fill_ring(Ops& ops, int first, int total, int step, int k_split, int kbs, int k_blocks) {
  constexpr int kStages = 4 * kGroups;
  int grp = 0;
  uint32_t parity = 0, filled = 0;
  bool ok = true;
  for (int unit = first; ok && unit < total && !ops.aborted(); unit += step) {
    const int kb0 = (unit % k_split) * kbs, kb1 = k_blocks < kb0 + kbs ? k_blocks : kb0 + kbs;
    ops.tile(unit / k_split);
    for (int kb = kb0; ok && kb < kb1; kb += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int stage = 4 * grp + i;
        if (ok && !ops.wait_empty(stage, parity ^ 1u)) ok = false;
        if (!ok) continue;
        ops.fill(stage, kb + i, kb + i < kb1);
        ++filled;
      }
      if (++grp == kGroups) {
        grp = 0;
        parity ^= 1u;
      }
    }
  }
  if (!ok) ops.abort();
  if (ops.aborted()) {   // no load may outlive the CTA's shared memory: each stage's last fill
    for (int s = 0; s < kStages; ++s) {
      const int last = ring_last_round(filled, s, kStages);
      if (last >= 0) ops.wait_full(s, (uint32_t)last & 1u);
    }
  }
}

}  // namespace csa
